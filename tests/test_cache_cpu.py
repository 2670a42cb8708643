"""Host side of the cache calls (hw_cache_write, hw_cache_read,
hw_block_commit_many_fp4, hw_block_move, hw_compact_moves): refusals, which come
before anything is enqueued, and the compaction's moves; and the 4-bit format's
reference against values worked by hand."""
import numpy as np
import pytest
import torch

from concurrent_shared_kv_gb300 import api, engine
from tests import fp4_ref as F

INVALID, UNSUPPORTED, CAPACITY, OVERLAP = -1, -2, -4, -5
A = 1 << 20  # an address that is never used: a refused call enqueues nothing


def status(f, *a, **kw):
    with pytest.raises(api.HwError) as e:
        f(*a, **kw)
    return e.value.status


def write(**kw):
    d = dict(dtype=api.HW_FP4_E2M1, n_layers=2, n_tokens=3, n_kv_heads=4, head_dim=128, rope_theta=1e6, k_new=A,
             v_new=2 * A, slot=3 * A, pos=4 * A, k_cache=5 * A, v_cache=6 * A, k_scale=0, v_scale=0, kv_scale=7 * A,
             capacity=100)
    d.update(kw)
    return api.cache_write(**{k: (v or None) if k in PTRS else v for k, v in d.items()}, stream=0)


def read(**kw):
    d = dict(dtype=api.HW_FP4_E2M1, n_layers=2, n_tokens=3, n_kv_heads=4, head_dim=128, k_cache=5 * A, v_cache=6 * A,
             k_scale=0, v_scale=0, kv_scale=7 * A, capacity=100, slot=3 * A, k_out=A, v_out=2 * A)
    d.update(kw)
    return api.cache_read(**{k: (v or None) if k in PTRS else v for k, v in d.items()}, stream=0)


PTRS = ("k_new", "v_new", "slot", "pos", "k_cache", "v_cache", "k_scale", "v_scale", "kv_scale", "k_out", "v_out", "flags")


@pytest.mark.parametrize("call", [write, read])
@pytest.mark.parametrize("kw,st", [
    (dict(dtype=7), INVALID), (dict(n_layers=-1), INVALID), (dict(n_tokens=-1), INVALID), (dict(n_kv_heads=0), INVALID),
    (dict(capacity=-1), INVALID), (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=64), UNSUPPORTED),
    (dict(dtype=api.HW_FP8_E4M3, head_dim=64), UNSUPPORTED), (dict(n_kv_heads=257), UNSUPPORTED),
    (dict(capacity=1 << 31), UNSUPPORTED), (dict(slot=0), INVALID), (dict(k_cache=0), INVALID), (dict(v_cache=0), INVALID),
    (dict(kv_scale=0), INVALID), (dict(dtype=api.HW_FP8_E4M3), INVALID), (dict(k_cache=5 * A + 8), INVALID),
    (dict(kv_scale=7 * A + 2), INVALID), (dict(slot=3 * A + 2), INVALID), (dict(flags=A + 1), INVALID)])
def test_cache_refusals(call, kw, st):
    assert status(call, **kw) == st


@pytest.mark.parametrize("call", [write, read])
@pytest.mark.parametrize("kw", [dict(k_scale=8 * A + 2), dict(v_scale=9 * A + 1)])
def test_head_scales_off_their_boundary(call, kw):
    """The heads' scales are read as floats: an address that is none is refused."""
    assert status(call, **dict(dict(dtype=api.HW_FP8_E4M3, k_scale=8 * A, v_scale=9 * A, kv_scale=0), **kw)) == INVALID


@pytest.mark.parametrize("kw", [dict(rope_theta=1.0), dict(rope_theta=float("nan")), dict(k_new=0), dict(v_new=0),
                                dict(pos=0), dict(k_new=A + 8), dict(pos=4 * A + 1)])
def test_write_refusals(kw):
    assert status(write, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(k_out=0), dict(v_out=0), dict(v_out=2 * A + 4)])
def test_read_refusals(kw):
    assert status(read, **kw) == INVALID


@pytest.mark.parametrize("call", [write, read])
@pytest.mark.parametrize("kw", [dict(n_tokens=0), dict(n_layers=0)])
def test_nothing_to_do(call, kw):
    assert call(slot=0, **kw) == 0


def commit(src=(0,), n=(4,), dst=(8,), delta=(3,), **kw):
    d = dict(n_layers=2, n_kv_heads=2, head_dim=128, rope_theta=1e4, k_src=A, v_src=2 * A, scale_src=3 * A,
             src_capacity=16, k_dst=4 * A, v_dst=5 * A, scale_dst=6 * A, dst_capacity=32)
    d.update(kw)
    return api.block_commit_many_fp4(**d, src_begin=src, n_tokens=n, dst_offset=dst, pos_delta=delta, stream=0)


@pytest.mark.parametrize("kw,st", [
    (dict(head_dim=64), UNSUPPORTED), (dict(rope_theta=0.5), INVALID), (dict(n=(-1,)), INVALID), (dict(src=(13,)), CAPACITY),
    (dict(dst=(29,)), CAPACITY), (dict(scale_src=None), INVALID), (dict(scale_dst=None), INVALID),
    (dict(scale_dst=6 * A + 2), INVALID), (dict(k_dst=4 * A + 8), INVALID),
    (dict(src=(0, 4), n=(4, 4), dst=(8, 11), delta=(0, 0)), OVERLAP),   # two destinations meet
    (dict(k_dst=A, dst_capacity=16), OVERLAP),                          # one pool for keys, and others for values
    (dict(scale_dst=3 * A), OVERLAP),                                   # scales of one cache, codes of two
    (dict(scale_dst=4 * A + 64), OVERLAP), (dict(scale_src=5 * A), OVERLAP), (dict(scale_dst=2 * A), OVERLAP),
    (dict(k_dst=A, v_dst=2 * A, scale_dst=3 * A, dst_capacity=16, dst=(2,)), OVERLAP)])  # a source is written over
def test_commit_refusals(kw, st):
    if kw == dict(k_dst=A, dst_capacity=16):
        kw = dict(kw, dst=(2,))
    assert status(commit, **kw) == st


@pytest.mark.parametrize("kw", [
    dict(k_dst=A, v_dst=2 * A),                     # one pool, scales of its tokens in two arrays
    dict(k_dst=A, scale_dst=3 * A),                 # keys in one pool, values in two
    dict(v_dst=2 * A, scale_dst=3 * A), dict(v_dst=2 * A), dict(k_dst=A),
    dict(k_dst=2 * A, v_dst=A), dict(k_dst=2 * A), dict(v_dst=A),  # keys among values
    dict(k_dst=2 * A, v_dst=A, scale_dst=3 * A)])
def test_commit_scales_belong_to_their_pool(kw):
    """The source's and the destination's scales are one array exactly where the pools are one."""
    assert status(commit, dst_capacity=16, **kw) == OVERLAP


def test_commit_of_nothing():
    assert commit(n=(0,), scale_src=None) == 0


def move(src=(0,), n=(4,), dst=(8,), **kw):
    d = dict(dtype=api.HW_BF16, n_layers=2, n_kv_heads=2, head_dim=128, k_cache=A, v_cache=2 * A, kv_scale=None,
             capacity=16)
    d.update(kw)
    return api.block_move(**d, src_begin=src, n_tokens=n, dst_begin=dst, stream=0)


@pytest.mark.parametrize("kw,st", [
    (dict(dtype=9), INVALID), (dict(n_kv_heads=0), INVALID), (dict(n_layers=-1), INVALID), (dict(capacity=-1), INVALID),
    (dict(head_dim=32), UNSUPPORTED), (dict(dtype=api.HW_FP4_E2M1, head_dim=64, kv_scale=3 * A), UNSUPPORTED),
    (dict(n=(-1,)), INVALID), (dict(src=(-1,)), INVALID), (dict(dst=(-2,)), INVALID), (dict(src=(13,)), CAPACITY),
    (dict(dst=(13,)), CAPACITY), (dict(k_cache=None), INVALID), (dict(v_cache=A + 16), OVERLAP),
    (dict(k_cache=A + 4), INVALID), (dict(kv_scale=3 * A), INVALID), (dict(dtype=api.HW_FP4_E2M1), INVALID),
    (dict(dtype=api.HW_FP4_E2M1, kv_scale=3 * A + 2), INVALID), (dict(dtype=api.HW_FP4_E2M1, kv_scale=A + 64), OVERLAP),
    (dict(src=(0,) * 257, n=(1,) * 257, dst=(1,) * 257), INVALID),
    (dict(capacity=1 << 31), UNSUPPORTED)])
def test_move_refusals(kw, st):
    assert status(move, **kw) == st


@pytest.mark.parametrize("kw", [dict(n=(0,)), dict(dst=(0,)), dict(src=(), n=(), dst=()), dict(n_layers=0)])
def test_moves_of_nothing(kw):
    assert move(**dict(dict(k_cache=None), **kw)) == 0


def test_move_status_needs_a_place():
    assert api.lib().hw_block_move_status(None, None) == INVALID


def test_sequences_of_unlike_lengths():
    with pytest.raises(ValueError):
        move(src=(0, 1))
    with pytest.raises(ValueError):
        commit(delta=(1, 2))


def test_numbers_past_32_bits():
    with pytest.raises(OverflowError):
        move(src=[1 << 32])
    for big in (np.array([1 << 32]), torch.tensor([(1 << 32) + 1]), np.array([0.5])):
        with pytest.raises(ValueError):
            move(src=big)


@pytest.mark.parametrize("bad", [[1.5], (0.5,), [np.float32(-0.5)], [torch.tensor(1.5)], [0, 2.000001], ["1"]])
def test_fractions_in_lists(bad):
    """Host sequences hold whole numbers, in lists as in arrays: nothing is cut."""
    some = [0] * len(bad)
    for args in ((bad, some, some), (some, bad, some), (some, some, bad)):
        with pytest.raises(ValueError):
            move(*args)
    with pytest.raises(ValueError):
        commit(src=some, n=some, dst=some, delta=bad)
    with pytest.raises(ValueError):
        api.compact_moves(bad, some, 10)
    whole = [float(x) for x in some]
    assert move(whole, some, some) == 0  # (a whole number may be a float)


def apply(pool, src, n, dst):
    for s, m, d in zip(src, n, dst):
        pool[d:d + m] = pool[s:s + m].copy()


@pytest.mark.parametrize("seed", range(40))
def test_compaction_keeps_every_block(seed):
    """Random blocks, empty ones among them, with and without room: the moves, one after
    the other, leave every block whole at its new start, in order and apart."""
    r = np.random.default_rng(seed)
    nb = int(r.integers(1, 12))
    lens = r.integers(0, 9, nb)
    starts, at = np.zeros(nb, np.int32), 0
    for b in r.permutation(nb):
        at += int(r.integers(0, 7))
        starts[b] = at
        at += int(lens[b])
    room = r.integers(0, 6, nb) if seed % 2 else None
    cap = max(at, int(lens.sum() + (0 if room is None else room.sum())))
    pool = np.arange(1000, 1000 + cap)
    held = [pool[s:s + m].copy() for s, m in zip(starts, lens)]
    new, src, n, dst = api.compact_moves(starts, lens, cap, room)
    apply(pool, src, n, dst)
    end = 0
    order = sorted(range(nb), key=lambda b: new[b] + 1e-3 * (lens[b] > 0))
    for b in order:
        assert np.array_equal(pool[new[b]:new[b] + lens[b]], held[b])
        assert new[b] >= end or lens[b] == 0
        end = max(end, new[b] + lens[b])
    assert list(np.sort(starts[lens > 0])) == [starts[b] for b in order if lens[b]]  # (the order is kept)


def test_compaction_by_hand():
    new, src, n, dst = api.compact_moves([10, 2, 20], [4, 3, 5], 40)
    assert new.tolist() == [3, 0, 7]
    assert (src.tolist(), n.tolist(), dst.tolist()) == ([2, 10, 20], [3, 4, 5], [0, 3, 7])
    new, src, n, dst = api.compact_moves([10, 2, 20], [4, 3, 5], 40, [0, 20, 0])  # the block at 2 keeps 20 free: two go up
    assert new.tolist() == [23, 0, 27]
    assert (src.tolist(), n.tolist(), dst.tolist()) == ([2, 20, 10], [3, 5, 4], [0, 27, 23])


@pytest.mark.parametrize("a,st", [
    (([0, 3], [4, 2], 10), OVERLAP), (([0, 8], [4, 3], 10), CAPACITY), (([-1], [1], 4), INVALID), (([0], [-1], 4), INVALID),
    (([0, 4], [4, 4], 10, [3, 0]), CAPACITY), (([0], [1], 4, [-1]), INVALID), (([0], [1], 1 << 31), UNSUPPORTED),
    ((list(range(257)), [1] * 257, 400), UNSUPPORTED)])
def test_compaction_refusals(a, st):
    assert status(api.compact_moves, *a) == st


def test_tensors_that_do_not_fit():
    """The engine's calls refuse what a kernel would read past, and tensors on the CPU."""
    k = torch.zeros(2, 3, 10, 64, dtype=torch.uint8)
    s = torch.zeros(2, 3, 10, 2, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    for kw in (dict(kv_scale=s[:, :, :9]), dict(kv_scale=s.float()), dict(kv_scale=s)):
        with pytest.raises(ValueError):
            engine.cache_read(i, k, k.clone(), **kw)
    with pytest.raises(ValueError):
        engine.block_move(k.to(torch.int16), k.to(torch.int16), [0], [1], [2])
    with pytest.raises(ValueError):
        engine.block_move(k, k[:, :, ::2], [0], [1], [2], kv_scale=s)


# ------------------------------------------------------- the format's reference

def test_levels_and_ties():
    codes = np.arange(16, dtype=np.uint8)
    assert F.decode(codes, np.float64(2)).tolist() == [0, 1, 2, 3, 4, 6, 8, 12, 0, -1, -2, -3, -4, -6, -8, -12]
    # a row whose scale is 1: borders go to the even code
    x = np.array([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5.0, -.25, -.75, .2500001, 5.000001, 0, -6, .1, 2.4])
    code, s = F.encode(x)
    assert s == 1 and code.tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 8, 10, 1, 7, 0, 15, 0, 4]
    assert np.array_equal(F.unpack(F.pack(code)), code) and F.pack(code)[0] == 0x07 and F.pack(code)[1] == 0x22


def test_scales():
    assert F.scale_of(np.zeros(4)) == 0 and F.scale_of(np.full(4, 6.0)) == 1
    assert F.scale_of(np.array([0, 2.0 ** -96])) > 0 and F.scale_of(np.array([0, 2.0 ** -99])) == 0
    assert np.isnan(F.scale_of(np.array([1, np.inf]))) and np.isnan(F.scale_of(np.array([1, np.nan])))
    assert np.isnan(F.scale_of(np.array([2.0 ** 100]))) and F.scale_of(np.array([2.0 ** 99])) > 0


def test_nearest_is_within_half_a_step():
    x = np.random.default_rng(0).standard_normal((200, 128)).astype(np.float32).astype(np.float64)
    code, s = F.encode(x)
    err = np.abs(F.decode(code, s) - x) / s[:, None]
    r = np.abs(x) / s[:, None]
    # half a step between levels; the largest element may stand up to the scale's rounding (2^-8 of 6) above 6
    assert (err <= np.where(r > 4, 1.0, np.where(r > 2, 0.5, 0.25)) + 1e-9).all()
