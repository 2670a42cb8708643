"""The cache calls on the GPU (hw_cache_write, hw_cache_read,
hw_block_commit_many_fp4, hw_block_move) against their definitions in 64 bits on
the host.

Tolerances, from the arithmetic: a rotated element is two fp32 products and a sum, off by
at most 3 * 2^-24 of |x0| + |x1|, and a cosine or sine by 2^-24 more (2^-21.4 of the
reduced angle's where it is a float of the turn): 2^-21 of |x0| + |x1| in all, kRot
below.  A stored element adds its type's half step: 2^-24, 2^-8 (bf16), 2^-4 (E4M3;
2^-10 where it is subnormal).  4 bits: the codes are the nearest ones except within kRot of
a border between two, and the scale is the nearest bf16 of max / 6 within as much."""
import numpy as np
import pytest
import torch

from concurrent_shared_kv_gb300 import api, engine
from tests import fp4_ref as F

pytestmark = pytest.mark.gpu

F32, BF16, FP8, FP4 = "f32", "bf16", "fp8", "fp4"
TORCH = {F32: torch.float32, BF16: torch.bfloat16, FP8: torch.float8_e4m3fn, FP4: torch.uint8}
ROT = 2.0 ** -21


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def new_tokens(g, layers, n, heads, d, dtype):
    act = torch.float32 if dtype == F32 else torch.bfloat16
    size = torch.exp(0.5 * torch.randn(layers, n, heads, 1, generator=g, device="cuda"))
    k = (torch.randn(layers, n, heads, d, generator=g, device="cuda") * size).to(act)
    v = (torch.randn(layers, n, heads, d, generator=g, device="cuda") * size.flip(1)).to(act)
    return k, v


def pools(layers, heads, cap, d, dtype, fill=None):
    """k_cache, v_cache and kv_scale (or None), bytes set to `fill` where given."""
    width = d // 2 if dtype == FP4 else d
    size = {F32: 4, BF16: 2}.get(dtype, 1)
    k, v = (torch.full((layers, heads, cap, width * size), 0 if fill is None else fill, dtype=torch.uint8,
                       device="cuda") for _ in range(2))
    k, v = k.view(TORCH[dtype]), v.view(TORCH[dtype])
    s = None
    if dtype == FP4:
        s = torch.full((layers, heads, cap, 4), 0 if fill is None else fill, dtype=torch.uint8,
                       device="cuda").view(torch.bfloat16)
    return k, v, s


def head_scales(x):
    return x.float().abs().amax(dim=(1, 3)).clamp(min=1e-20) / 448.0  # [layers, heads]


def check_codes(y, size, packed, s):
    """4-bit rows [..., 64] under s [...] hold y [..., 128] (64 bits), whose fp32
    counterpart is off by at most ROT * size (size [...]: what |x0| + |x1| reach)."""
    y, s = np.asarray(y), np.asarray(s)
    top = np.abs(y).max(-1)
    off = ROT * size
    assert (np.abs(s - top / 6) <= top / 6 * 2.0 ** -8 / (1 + 2.0 ** -8) * 1.0001 + off / 6).all()
    live = s > 0
    codes = F.unpack(packed)
    assert (codes[~live] == 0).all()
    r = np.abs(y[live]) / s[live][:, None]
    slack = (off[live] / s[live])[:, None]
    low = np.concatenate([[0.0], (F.LEVELS[1:] + F.LEVELS[:-1]) / 2])  # a code's range
    high = np.concatenate([(F.LEVELS[1:] + F.LEVELS[:-1]) / 2, [np.inf]])
    c = codes[live] & 7
    assert (r >= low[c] - slack).all() and (r <= high[c] + slack).all()
    wrong = (codes[live] >= 8) != (y[live] < 0)
    assert (np.abs(y[live])[wrong] <= (off[live][:, None] + 0 * r)[wrong]).all()


def check_written(dtype, y, size, cache, scale, d):
    """cache [...] of one pool against y [..., D]; scale: the heads' or the tokens'."""
    off = ROT * size[..., None]
    if dtype == FP4:
        return check_codes(y, size, cache, scale)
    if dtype == FP8:
        got = cache * scale[..., None]
        z = np.clip(y / scale[..., None], -448, 448)
        tol = np.maximum(np.abs(z) * 2.0 ** -4, 2.0 ** -10) + 448 * 2.0 ** -22
        assert (np.abs(got - z * scale[..., None]) <= tol * scale[..., None] + off).all()
    else:
        assert (np.abs(cache - y) <= np.abs(y) * (2.0 ** -24 if dtype == F32 else 2.0 ** -8) + off).all()


SHAPES = [  # layers, tokens, heads, D
    (1, 1, 1, 128), (1, 4, 8, 128), (3, 17, 2, 64), (2, 16, 5, 128), (1, 333, 8, 64), (7, 33, 3, 128), (2, 1500, 8, 128)]


@pytest.mark.parametrize("dtype", [F32, BF16, FP8, FP4])
@pytest.mark.parametrize("layers,n,heads,d", SHAPES)
def test_write_and_read(dtype, layers, n, heads, d):
    if d == 64 and dtype in (FP8, FP4):
        pytest.skip("8 and 4 bits: head_dim 128")
    g = gen(n + heads)
    k_new, v_new = new_tokens(g, layers, n, heads, d, dtype)
    cap = 2 * n + 5
    k, v, s = pools(layers, heads, cap, d, dtype, fill=0x3c)
    k0, v0, s0 = (None if x is None else x.clone() for x in (k, v, s))
    slot = torch.randperm(cap, generator=g, device="cuda")[:n].int()
    pos = torch.randint(0, 70000, (n,), generator=g, device="cuda").int()
    if n > 3:
        slot[2] = -1  # left out
        pos[1], pos[3] = -5, 2 ** 31 - 1
    ks, vs = (head_scales(k_new), head_scales(v_new)) if dtype == FP8 else (None, None)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    engine.cache_write(k_new, v_new, slot, pos, k, v, rope_theta=1e6, k_scale=ks, v_scale=vs, kv_scale=s, flags=flags)
    k_out, v_out = engine.cache_read(slot, k, v, k_scale=ks, v_scale=vs, kv_scale=s, flags=flags)
    assert flags.item() == 0
    on = (slot >= 0).nonzero()[:, 0]
    at = slot[on].long()
    rest = torch.ones(cap, dtype=torch.bool, device="cuda")
    rest[at] = False
    for x, x0 in ((k, k0), (v, v0), (s, s0)):  # nothing else is written
        if x is not None:
            assert torch.equal(x.view(torch.uint8)[:, :, rest], x0.view(torch.uint8)[:, :, rest])
    x = k_new[:, on].double().cpu().numpy()
    want = {"k": F.rotate(x, pos[on].cpu().numpy()[:, None], 1e6), "v": v_new[:, on].double().cpu().numpy()}
    half = d // 2
    pair = np.abs(x[..., :half]) + np.abs(x[..., half:])
    for name, cache, hs, out in (("k", k, ks, k_out), ("v", v, vs, v_out)):
        y = want[name]  # [layers, n, heads, D]
        size = pair.max(-1) * (name == "k")
        # (angles of far positions: this reference's own 2^-53 of a turn count)
        size = size * (1 + np.abs(pos[on].cpu().numpy()).astype(np.float64) * 2.0 ** -30)[:, None]
        got = cache[:, :, at].transpose(1, 2)
        if dtype == FP4:
            scale = s[:, :, at, 0 if name == "k" else 1].transpose(1, 2)
            check_written(dtype, y, size, got.cpu().numpy(), scale.double().cpu().numpy(), d)
            value = F.values(got, scale)
        else:
            scale = None if hs is None else hs[:, None].expand(layers, len(on), heads).double().cpu().numpy()
            check_written(dtype, y, size, got.double().cpu().numpy(), scale, d)
            value = got.double().cpu().numpy() * (1 if scale is None else scale[..., None])
        # read back: the value in fp32 (codes times scales are at most 24 bits), rounded once
        value = torch.tensor(value).float().to(out.dtype)
        assert torch.equal(out[:, on].cpu(), value)


@pytest.mark.parametrize("dtype", [BF16, FP8, FP4])
def test_written_as_appended(dtype):
    """A token has the same bits whether hw_cache_write stores it or a decode call
    appends it."""
    g = gen(5)
    heads, cap, rows = 4, 300, 3
    k_new, v_new = new_tokens(g, 1, rows, heads, 128, dtype)
    k1, v1, s1 = pools(1, heads, cap, 128, dtype)
    k2, v2, s2 = pools(1, heads, cap, 128, dtype)
    ks, vs = (head_scales(k_new), head_scales(v_new)) if dtype == FP8 else (None, None)
    starts, lens = [0, 100, 200], [77, 100, 1]
    pos = torch.tensor([n - 1 for n in lens], dtype=torch.int32, device="cuda")
    slot = pos + torch.tensor(starts, dtype=torch.int32, device="cuda")
    engine.cache_write(k_new, v_new, slot, pos, k1, v1, rope_theta=1e4, k_scale=ks, v_scale=vs, kv_scale=s1)
    t = engine.DecodeSession(n_rows=rows, n_q_heads=8, n_kv_heads=heads, head_dim=128, n_blocks=3, max_view_blocks=1,
                             capacity=cap, dtype=torch.bfloat16, rope_theta=1e4, kv_fp8=dtype == FP8,
                             kv_fp4=dtype == FP4)
    t.set_metadata(starts, lens, [[0], [1], [2]], [[0], [0], [0]], pos)
    t.plan_append([0, 1, 2], pos)
    q = torch.randn(rows, 8, 128, generator=g, device="cuda").to(torch.bfloat16)
    if dtype == FP4:
        t.append_decode_planned_fp4(q, k_new, v_new, k2, v2, s2)
    elif dtype == FP8:
        t.append_decode_planned_fp8(q, k_new, v_new, k2, v2, ks, vs)
    else:
        t.append_decode_planned(q, k_new, v_new, k2, v2)
    assert t.device_flags() == 0
    for a, b in ((k1, k2), (v1, v2), (s1, s2)):
        assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_write_values_at_the_edges():
    """Zeros, ties, tiny, huge and non-finite tokens in 4 bits, at position 0 (no turn)."""
    rows = np.zeros((12, 128), np.float32)
    rows[1] = 6.0
    rows[2, :16] = [6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5.0, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5.0, -6]
    rows[3] = 2.0 ** -102                      # below the format: zero
    rows[4, 5] = 2.0 ** -97                    # just in
    rows[5, 127] = 2.0 ** 99
    rows[6, 64] = 2.0 ** 100                   # out: NaN
    rows[7, 3], rows[8, 100], rows[9, 0] = np.inf, -np.inf, np.nan
    rows[10] = np.linspace(-3, 3, 128)
    rows[11, 31] = -7.0
    x = torch.tensor(rows).to(torch.bfloat16).cuda().reshape(1, 12, 1, 128)
    n = x.shape[1]
    k, v, s = pools(1, 1, n, 128, FP4, fill=0xff)
    slot = torch.arange(n, dtype=torch.int32, device="cuda")
    engine.cache_write(x, x, slot, torch.zeros_like(slot), k, v, rope_theta=1e4, kv_scale=s)
    want, scale = F.encode(x[0, :, 0].double().cpu().numpy())
    for cache, i in ((k, 0), (v, 1)):
        assert np.array_equal(s[0, 0, :, i].double().cpu().numpy(), scale, equal_nan=True)
        assert np.array_equal(F.unpack(cache[0, 0].cpu().numpy()) & 7, want & 7)
        assert np.array_equal(F.decode(F.unpack(cache[0, 0].cpu().numpy()), scale), F.decode(want, scale), equal_nan=True)
    k_out, _ = engine.cache_read(slot, k, v, kv_scale=s)
    bad = torch.isnan(k_out[0, :, 0]).all(-1)
    assert bad.tolist() == [i in (6, 7, 8, 9) for i in range(n)]


def test_slots_out_of_range():
    """Tokens whose slot is none are left out, on both ways, and reported."""
    g = gen(1)
    k_new, v_new = new_tokens(g, 2, 5, 2, 128, BF16)
    k, v, _ = pools(2, 2, 8, 128, BF16)
    slot = torch.tensor([3, 8, -2, -1, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    pos = torch.zeros_like(slot)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    engine.cache_write(k_new, v_new, slot, pos, k, v, rope_theta=1e4, flags=flags)
    assert flags.item() == 2  # HW_DEV_BAD_RANGE
    assert torch.equal(v[:, :, 3], v_new[:, 0]) and torch.equal(k[:, :, 3], k_new[:, 0])
    assert k.view(torch.int16).count_nonzero() <= 2 * 2 * 128
    flags.zero_()
    out = torch.full((2, 5, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    k_out, v_out = engine.cache_read(slot, k, v, k_out=out, v_out=out.clone(), flags=flags)
    assert flags.item() == 2
    assert torch.equal(v_out[:, 0], v_new[:, 0]) and (k_out[:, 1:] == 7).all() and (v_out[:, 1:] == 7).all()
    flags.zero_()
    engine.cache_read(slot[[0, 3]], k, v, flags=flags)  # -1 alone is no error
    engine.cache_write(k_new[:, :2].contiguous(), v_new[:, :2].contiguous(), slot[[0, 3]], pos[:2], k, v, rope_theta=1e4, flags=flags)
    assert flags.item() == 0


# ------------------------------------------------------------------- commits

@pytest.mark.parametrize("layers,heads,commits", [
    (1, 1, [(0, 1, 3, 3)]), (2, 3, [(5, 37, 11, 1001)]), (3, 2, [(0, 20, 40, -7), (30, 1, 0, 65000), (31, 9, 60, 0)]),
    (4, 8, [(0, 300, 100, 16384)]),
    (8, 8, [(0, 200, 0, 7), (200, 0, 200, 5), (200, 65, 200, -9), (265, 55, 340, 0)])])  # CTAs that cross ranges
def test_commit(layers, heads, commits):
    g = gen(heads)
    cs, cd = 320, 400
    kp, ks = F.draw(g, layers, heads, cs, 128)
    vp, vs = F.draw(g, layers, heads, cs, 128)
    if layers == 2:
        ks[0, 1, 7], vs[1, 0, 8] = float("nan"), float("nan")  # tokens that are not finite stay so
        kp[0, 1, 7] = 0
    scale = torch.stack([ks, vs], -1)
    kd, vd, sd = pools(layers, heads, cd, 128, FP4, fill=0x11)
    k0, v0, s0 = kd.clone(), vd.clone(), sd.clone()
    engine.block_commit_fp4(kp, vp, scale, kd, vd, sd, *zip(*commits), rope_theta=1e6)
    rest = torch.ones(cd, dtype=torch.bool, device="cuda")
    for src, n, dst, delta in commits:
        rest[dst:dst + n] = False
        assert torch.equal(vd[:, :, dst:dst + n], vp[:, :, src:src + n])
        assert torch.equal(sd[:, :, dst:dst + n, 1].view(torch.int16), scale[:, :, src:src + n, 1].view(torch.int16))
        got, gs = kd[:, :, dst:dst + n].cpu().numpy(), sd[:, :, dst:dst + n, 0].double().cpu().numpy()
        if delta == 0:
            assert torch.equal(kd[:, :, dst:dst + n], kp[:, :, src:src + n])
            assert torch.equal(sd[:, :, dst:dst + n, 0], scale[:, :, src:src + n, 0])
            continue
        x = F.values(kp[:, :, src:src + n], ks[:, :, src:src + n])
        y = F.rotate(x, np.float64(delta), 1e6)
        ok = np.isfinite(x).all(-1)
        assert np.array_equal(np.isnan(gs), ~ok)
        size = (np.abs(x[..., :64]) + np.abs(x[..., 64:])).max(-1)
        check_codes(y[ok], size[ok], got[ok], gs[ok])
    for x, x0 in ((kd, k0), (vd, v0), (sd, s0)):
        assert torch.equal(x.view(torch.uint8)[:, :, rest], x0.view(torch.uint8)[:, :, rest])


def test_commit_within_a_pool():
    g = gen(3)
    kp, ks = F.draw(g, 2, 2, 64, 128)
    vp, vs = F.draw(g, 2, 2, 64, 128)
    s = torch.stack([ks, vs], -1)
    kd, vd, sd = (x.clone() for x in (kp, vp, s))
    engine.block_commit_fp4(kp, vp, s, kd, vd, sd, [3], [20], [40], [9], rope_theta=1e4)
    engine.block_commit_fp4(kp, vp, s, kp, vp, s, [3], [20], [40], [9], rope_theta=1e4)
    for a, b in ((kp, kd), (vp, vd), (s, sd)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# --------------------------------------------------------------------- moves

def moved(x, src, n, dst):
    x = x.clone()
    for s, m, d in zip(src, n, dst):
        x[:, :, d:d + m] = x[:, :, s:s + m].clone()
    return x


MOVES = {  # src, n, dst over a pool of 700 tokens
    "copy": ([10], [100], [400]),
    "fork": ([3] * 4, [129] * 4, [140, 270, 400, 530]),
    "down by one": ([1], [699], [0]),
    "up by one": ([0], [699], [1]),
    "down far": ([300], [400], [5]),
    "up far": ([2], [500], [190]),
    "compact": ([7, 150, 300, 650], [100, 129, 200, 50], [0, 100, 229, 429]),
    "swap through a third": ([0, 100, 400], [100, 100, 100], [400, 0, 100]),
    "chain": ([0, 200, 400], [150, 150, 150], [200, 400, 550]),     # each reads what the one before wrote
    "same place twice": ([0, 200], [120, 130], [400, 410]),         # the later one stands
    "over a source": ([100, 0], [50, 120], [600, 90]),              # the second writes where the first has read
    "nothing and itself": ([5, 9, 0], [0, 30, 20], [100, 9, 60]),
    "single tokens": ([699, 0, 350], [1, 1, 1], [0, 699, 351]),
}


@pytest.mark.parametrize("dtype,d", [(F32, 64), (F32, 128), (BF16, 64), (BF16, 128), (FP8, 128), (FP4, 128)])
@pytest.mark.parametrize("what", MOVES)
def test_moves(what, dtype, d):
    g = gen(11)
    k, v, s = pools(2, 3, 700, d, dtype)
    for x in (k, v) + (() if s is None else (s,)):
        x.view(torch.uint8).random_(0, 256, generator=g)
    src, n, dst = MOVES[what]
    want = [None if x is None else moved(x.view(torch.uint8), src, n, dst) for x in (k, v, s)]
    engine.block_move(k, v, src, n, dst, kv_scale=s)
    for x, w in zip((k, v, s), want):
        assert x is None or torch.equal(x.view(torch.uint8), w)


@pytest.mark.parametrize("layers,heads,dtype", [(1, 1, BF16), (40, 8, FP4), (5, 8, F32)])
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_many_moves(layers, heads, dtype, seed):
    """Random sequences of up to 256 moves that meet one another in every way, and a
    few that do not, on few rows and on more rows than CTAs."""
    r = np.random.default_rng(seed)
    cap = 5000 if layers == 1 else 900
    m = int(r.integers(1, 257)) if seed else 256
    n = r.integers(0, 200, m)
    src = np.array([r.integers(0, cap - x + 1) for x in n])
    dst = np.array([r.integers(0, cap - x + 1) for x in n])
    k, v, s = pools(layers, heads, cap, 128, dtype)
    g = gen(seed)
    for x in (k, v) + (() if s is None else (s,)):
        x.view(torch.uint8).random_(0, 256, generator=g)
    want = [None if x is None else moved(x.view(torch.uint8), src, n, dst) for x in (k, v, s)]
    engine.block_move(k, v, src, n, dst, kv_scale=s)
    for x, w in zip((k, v, s), want):
        assert x is None or torch.equal(x.view(torch.uint8), w)


def test_long_slide():
    """A block of many chunks by less than a chunk, both ways."""
    k = torch.randint(0, 1 << 15, (1, 2, 60000, 128), dtype=torch.int16, device="cuda").view(torch.bfloat16)
    v = torch.randint(0, 1 << 15, (1, 2, 60000, 128), dtype=torch.int16, device="cuda").view(torch.bfloat16)
    for src, dst in ((13, 0), (0, 13), (70, 5)):
        want = [moved(x.view(torch.int16), [src], [59900], [dst]) for x in (k, v)]
        engine.block_move(k, v, [src], [59900], [dst])
        assert torch.equal(k.view(torch.int16), want[0]) and torch.equal(v.view(torch.int16), want[1])


def test_compact_keeps_blocks():
    g = gen(2)
    k, ks = F.draw(g, 3, 2, 500, 128)
    v, vs = F.draw(g, 3, 2, 500, 128)
    s = torch.stack([ks, vs], -1)
    starts, lens, room = [40, 300, 120, 0], [60, 128, 100, 0], [0, 0, 150, 5]
    held = [[x[:, :, a:a + n].clone() for a, n in zip(starts, lens)] for x in (k, v, s)]
    new = engine.compact(k, v, starts, lens, room=room, kv_scale=s)
    assert new.tolist() == [5, 315, 65, 0]
    for x, h in zip((k, v, s), held):
        for a, n, b in zip(new.tolist(), lens, h):
            assert torch.equal(x[:, :, a:a + n].view(torch.uint8), b.view(torch.uint8))


# --------------------------------------------------- streams, graphs, devices

def test_on_a_stream_and_in_a_graph():
    """Each call runs on the stream it is given, and can be captured and replayed."""
    g = gen(9)
    k_new, v_new = new_tokens(g, 2, 40, 3, 128, FP4)
    k, v, s = pools(2, 3, 200, 128, FP4)
    slot = torch.arange(40, dtype=torch.int32, device="cuda")
    out = [torch.zeros(2, 40, 3, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def all_calls(stream):
        engine.cache_write(k_new, v_new, slot, slot, k, v, rope_theta=1e4, kv_scale=s, stream=stream)
        engine.block_move(k, v, [0, 0], [40, 40], [40, 80], kv_scale=s, stream=stream)
        engine.block_commit_fp4(k, v, s, k, v, s, [80], [40], [120], [50], rope_theta=1e4, stream=stream)
        engine.cache_read(slot + 120, k, v, kv_scale=s, k_out=out[0], v_out=out[1], stream=stream)

    with torch.cuda.stream(side):
        all_calls(side)
    side.synchronize()
    want = [x.clone() for x in out]
    assert want[0].abs().sum() > 0
    at = slot + 120
    for x in (k, v, s, *out):
        x.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        engine.cache_write(k_new, v_new, slot, slot, k, v, rope_theta=1e4, kv_scale=s)
        engine.block_move(k, v, [0, 0], [40, 40], [40, 80], kv_scale=s)
        engine.block_commit_fp4(k, v, s, k, v, s, [80], [40], [120], [50], rope_theta=1e4)
        engine.cache_read(at, k, v, kv_scale=s, k_out=out[0], v_out=out[1])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_tensors_that_do_not_fit():
    k, v, s = pools(1, 2, 10, 128, FP4)
    i = torch.zeros(4, dtype=torch.int32, device="cuda")
    x = torch.zeros(1, 4, 2, 128, dtype=torch.bfloat16, device="cuda")
    ok = dict(rope_theta=1e4, kv_scale=s)
    engine.cache_write(x, x, i - 1, i, k, v, **ok)
    for bad in ((x.float(), x, i, i, k, v), (x[:, :3], x, i, i, k, v), (x, x, i.long(), i, k, v), (x, x, i, i[:3], k, v),
                (x, x, i, i, k, v[:, :1]), (x, x, i.cpu(), i, k, v), (x, x, i, i, k.view(torch.float8_e4m3fn), v)):
        with pytest.raises(ValueError):
            engine.cache_write(*bad, **ok)
    with pytest.raises(ValueError):
        engine.cache_write(x, x, i, i, k, v, rope_theta=1e4)  # bytes without kv_scale: E4M3, whose scales are missing
    with pytest.raises(ValueError):
        engine.cache_read(i, k, v, kv_scale=s, k_out=x[:, :2])
    with pytest.raises(ValueError):
        engine.block_commit_fp4(k, v, s, *pools(2, 2, 10, 128, FP4), [0], [1], [5], [1], rope_theta=1e4)


def test_offsets_past_32_bits():
    """Pools whose last tokens lie past 2^32 bytes and 2^31 elements."""
    cap = 9_000_000
    k, v, s = pools(1, 4, cap, 128, FP4)  # 2.3 GB each
    g = gen(4)
    x, y = new_tokens(g, 1, 33, 4, 128, FP4)
    slot = torch.arange(cap - 33, cap, dtype=torch.int32, device="cuda")
    engine.cache_write(x, y, slot, slot, k, v, rope_theta=1e6, kv_scale=s)
    small = pools(1, 4, 33, 128, FP4)
    near = torch.arange(33, dtype=torch.int32, device="cuda")
    engine.cache_write(x, y, near, slot, *small[:2], rope_theta=1e6, kv_scale=small[2])
    for a, b in zip((k, v, s), small):
        assert torch.equal(a[:, :, -33:].view(torch.uint8), b.view(torch.uint8))
    got = engine.cache_read(slot, k, v, kv_scale=s)
    want = engine.cache_read(near, *small[:2], kv_scale=small[2])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    engine.block_move(k, v, [cap - 33], [33], [7], kv_scale=s)
    engine.block_commit_fp4(k, v, s, k, v, s, [cap - 33], [33], [100], [0], rope_theta=1e6)
    for a, b in zip((k, v, s), small):
        for at in (7, 100):
            assert torch.equal(a[:, :, at:at + 33].view(torch.uint8), b.view(torch.uint8))


def near_ties(n, seed):
    """Numbers of bf16 and an fp32 scale each, whose quotient lies as near to a border between
    two E4M3 codes as fp32 allows."""
    r = np.random.default_rng(seed)
    x = torch.tensor(r.standard_normal(n), dtype=torch.float32).bfloat16().float()
    border = (17 + 2 * torch.tensor(r.integers(0, 8, n))) / 16.0 * 2.0 ** torch.tensor(r.integers(-5, 8, n))
    return x, (x.abs().double() / border.double()).float()


def test_e4m3_tokens_are_divided():
    """Codes are those of the quotient by the head's scale (fp32, as the decode reads
    them), whether written or appended: not of a product with the reciprocal."""
    heads = 128
    x, s = near_ties(40 * heads, 3)
    want = (x / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    other = (x * (1 / s)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    assert (want != other).sum() > 100  # (the inputs tell the two apart)
    x, s, want = x.view(40, heads, 1).cuda(), s.view(40, heads).cuda(), want.view(40, heads, 1).cuda()
    new = x.expand(40, heads, 128).bfloat16().contiguous()[:, None]  # [layers][1][heads][128]
    k, v, _ = pools(40, heads, 2, 128, FP8)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    engine.cache_write(new, new, zero, zero, k, v, rope_theta=1e4, k_scale=s, v_scale=s)
    for pool in (k, v):  # (position 0: keys are not turned)
        assert torch.equal(pool[:, :, 0].view(torch.uint8), want.expand(40, heads, 128))
    t = engine.DecodeSession(n_rows=1, n_q_heads=heads, n_kv_heads=heads, head_dim=128, n_blocks=1, max_view_blocks=1,
                             capacity=2, dtype=torch.bfloat16, rope_theta=1e4, kv_fp8=True)
    t.set_metadata([0], [1], [[0]], [[0]], [0])
    t.plan_append([0], [0])
    for l in range(40):
        k, v, _ = pools(1, heads, 2, 128, FP8)
        t.append_decode_planned_fp8(new[l], new[l], new[l], k, v, s[l], s[l])
        for pool in (k, v):
            assert torch.equal(pool[0, :, 0].view(torch.uint8), want[l].expand(heads, 128))
    assert t.device_flags() == 0


def test_e4m3_saturates_at_any_scale():
    """Quotients past 448 are 448, infinities among them, at scales from 2^-126 to 2^126; NaN stays NaN."""
    scales = torch.tensor([2.0 ** -126, 2.0 ** -90, 1.7, 2.0 ** 90, 1.3 * 2.0 ** 126], device="cuda")
    rows = []
    for s in scales.double().tolist():
        a = torch.linspace(-500, 500, 128, dtype=torch.float64) * s
        a[:8] = torch.tensor([np.inf, -np.inf, np.nan, 3e38, -3e38, 0.0, 2.0 ** -126, s])
        rows.append(a.clamp(-3.3e38, 3.3e38).where(a.abs() < np.inf, a).to(torch.bfloat16))
    v_new = torch.stack(rows)[None].cuda().contiguous()  # [1 token][5 heads][128]
    k, v, _ = pools(1, 5, 3, 128, FP8, fill=0)
    at = torch.ones(1, dtype=torch.int32, device="cuda")
    engine.cache_write(v_new, v_new, at, at - 1, k[0], v[0], rope_theta=1e4, k_scale=scales, v_scale=scales)
    q = (v_new[0].float() / scales[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    got = v[0, :, 1]
    assert torch.equal(torch.isnan(got.float()), torch.isnan(q.float())) and torch.isnan(got.float()).sum() == 5
    same = ~torch.isnan(q.float())
    assert torch.equal(got.view(torch.uint8)[same], q.view(torch.uint8)[same])


def turned_in_32_bits(x, delta, theta):
    """x [..., 128] fp32 turned as the format defines it: cosines and sines rounded to fp32, every
    product and sum rounded."""
    a = np.float64(delta) * np.float64(theta) ** (-np.arange(64) / 64)
    c, s = np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)
    lo, hi = x[..., :64], x[..., 64:]
    return np.concatenate([lo * c - hi * s, hi * c + lo * s], -1)


def encoded(y):
    """(codes, scales) of fp32 rows: the nearest levels of the exact quotients, ties to the even code."""
    top = np.abs(y).max(-1)
    scale = F.bf16(top * np.float32(1 / 6))
    r = np.abs(y).astype(np.float64)[..., None]
    border = (F.LEVELS[1:] + F.LEVELS[:-1]) / 2 * scale[..., None, None]  # (exact: 3 bits times 8)
    even_below = np.arange(7) % 2 == 0
    code = np.where(even_below, r > border, r >= border).sum(-1)
    return (code + 8 * np.signbit(y)).astype(np.uint8), scale


def tie_rows(delta, theta):
    """Keys whose last pair is not turned in 32 bits and stands, under the new scale that the first
    pair makes, at a border between two levels."""
    rows, scales = [], []
    for m in range(128, 256):
        s = np.float32(m / 128)
        for a in range(16):
            for b in range(8):
                codes = np.zeros(128, np.uint8)
                codes[0], codes[64] = a, b
                _, nxt = encoded(turned_in_32_bits(F.decode(codes, s).astype(np.float32), delta, theta))
                for level in range(1, 8):
                    tie = F.LEVELS[level] * np.float64(s) / max(nxt, 1e-9)
                    if tie in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
                        codes[63] = level
                        if encoded(turned_in_32_bits(F.decode(codes, s).astype(np.float32), delta, theta))[1] == nxt:
                            rows.append(codes.copy())
                            scales.append(s)
    return np.array(rows), np.array(scales)


@pytest.mark.parametrize("delta,theta", [(1, 1e6), (7, 1e6), (-100, 1e7), (40, 1e7)])
def test_commits_decide_borders(delta, theta):
    """A committed key is the stored one decoded, turned in 32 bits, and encoded: exactly at borders
    between levels (ties to the even code), and but for 2^-21 beside them (the turn's
    roundings, in whatever order they are made)."""
    codes, scales = tie_rows(delta, theta)
    assert len(codes) > 50
    g = gen(17)
    more, ms = F.draw(g, 3000, 128)
    n = len(codes) + 3000
    packed = torch.cat([torch.tensor(F.pack(codes)).cuda(), more])[None, None].contiguous()
    ks = torch.cat([torch.tensor(scales).cuda().bfloat16(), ms])
    scale = torch.stack([ks, torch.ones_like(ks)], -1)[None, None].contiguous()
    kd, vd, sd = pools(1, 1, n, 128, FP4)
    engine.block_commit_fp4(packed, packed, scale, kd, vd, sd, [0], [n], [0], [delta], rope_theta=theta)
    y = turned_in_32_bits(F.values(packed[0, 0], ks).astype(np.float32), delta, theta)
    want, want_scale = encoded(y)
    got, got_scale = F.unpack(kd[0, 0].cpu().numpy()), sd[0, 0, :, 0].double().cpu().numpy()
    same = got_scale == want_scale
    assert same[:len(codes)].all() and same.mean() > 0.999
    border = (F.LEVELS[1:] + F.LEVELS[:-1]) / 2 * want_scale[:, None, None]
    size = (np.abs(y[:, :64]) + np.abs(y[:, 64:])).max(-1)[:, None]
    beside = (np.abs(np.abs(y)[..., None] - border) <= 2.0 ** -21 * size[..., None]).any(-1)
    beside[:len(codes), 63] = False  # (ties)
    assert beside.mean() < 1e-3
    wrong = F.decode(got, want_scale) != F.decode(want, want_scale)
    assert not (wrong & ~beside)[same].any()


def test_moves_have_a_status():
    """A move whose copies all land leaves no error bit, ordered or not, on any stream."""
    k, v, s = pools(2, 3, 700, 128, FP4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for src, n, dst in MOVES.values():
        engine.block_move(k, v, src, n, dst, kv_scale=s, stream=side)
    assert api.block_move_status(stream=side) == 0 and api.block_move_status() == 0


def test_e4m3_keys_turn_as_precisely_as_32_bits_can():
    """Of 10^8 keys no more have another code than the 64-bit rotation gives than where
    cosines, sines, products and sums are rounded to fp32 and nothing else is: both counts are of
    independent, rare events, so three deviations of their difference are allowed."""
    heads, n, theta = 8, 12500, 1e6
    freq = theta ** (-torch.arange(64, dtype=torch.float64, device="cuda") / 64)
    ours = plain = 0
    for seed in range(8):
        g = gen(seed)
        x = torch.randn(1, n, heads, 128, generator=g, device="cuda").bfloat16()
        pos = torch.randint(0, 70000, (n,), generator=g, device="cuda").int()
        s = head_scales(x)
        k, v, _ = pools(1, heads, n, 128, FP8)
        slot = torch.arange(n, dtype=torch.int32, device="cuda")
        engine.cache_write(x, x, slot, pos, k, v, rope_theta=theta, k_scale=s, v_scale=s)

        def codes(dtype):
            a = pos.double()[:, None, None] * freq
            c, sn = a.cos().to(dtype), a.sin().to(dtype)
            lo, hi = x[0, ..., :64].to(dtype), x[0, ..., 64:].to(dtype)
            y = torch.cat([lo * c - hi * sn, hi * c + lo * sn], -1) / s[0].to(dtype)[:, None]
            return y.float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        want = codes(torch.float64)
        ours += (k[0].view(torch.uint8).transpose(0, 1) != want).sum().item()
        plain += (codes(torch.float32) != want).sum().item()
    assert plain > 50 and ours <= plain + 3 * (2 * plain) ** 0.5, (ours, plain)
