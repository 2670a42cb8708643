"""Decode over 4-bit caches without a GPU: the argument checks, which run before
anything is enqueued, and which calls refuse a 4-bit description."""
import ctypes

import pytest
import torch

from concurrent_shared_kv_gb300 import api, engine

A = 1 << 20  # an address that is never used: a refused call enqueues nothing
INVALID, UNSUPPORTED = -1, -2


def desc(**kw):
    base = dict(n_rows=2, n_q_heads=4, n_kv_heads=2, head_dim=128, n_blocks=3, max_view_blocks=3,
                cache_capacity=400, dtype=api.HW_FP4_E2M1, rope_theta=1e6, scale=0.088)
    base.update(kw)
    return api.make_desc(**base)


def status(fn, *args, **kw):
    with pytest.raises(api.HwError) as e:
        fn(*args, **kw)
    return e.value.status


def decode(d, s=A):
    return status(api.attn_decode_planned_fp4, d, A, A, A, s, A, None, A, 0)


def append(d, s=A):
    return status(api.attn_append_decode_planned_fp4, d, A, A, A, A, A, s, A, None, A, 0)


@pytest.mark.parametrize("call", [decode, append])
def test_entry_checks(call):
    assert call(desc(), s=None) == INVALID
    assert call(desc(), s=A + 2) == INVALID  # a token's scales are one 4-byte word
    for other in (api.HW_BF16, api.HW_F32, api.HW_FP8_E4M3):
        assert call(desc(dtype=other)) == INVALID  # another cache: its own call
    assert call(desc(head_dim=64)) == UNSUPPORTED
    assert call(desc(dtype=7)) == INVALID
    # past the checks of the description (and stopped at the workspace, which needs a device)
    assert call(desc()) not in (INVALID, UNSUPPORTED)


def test_appends_take_no_limits():
    assert append(desc(flags=api.HW_DESC_VIEW_LIMITS)) == UNSUPPORTED
    assert decode(desc(flags=api.HW_DESC_VIEW_LIMITS)) not in (INVALID, UNSUPPORTED)


def test_the_other_calls_refuse_the_description():
    d = desc()
    assert status(api.attn_decode, d, A, A, A, A, A, A, A, A, A, None, A, 0) == UNSUPPORTED
    assert status(api.attn_decode_noalloc, d, A, A, A, A, A, A, A, A, A, None) == UNSUPPORTED
    assert status(api.attn_decode_planned, d, A, A, A, A, None, A, 0) == UNSUPPORTED
    assert status(api.attn_append_decode_planned, d, A, A, A, A, A, A, None, A, 0) == UNSUPPORTED
    assert status(api.attn_decode_planned_fp8, d, A, A, A, A, A, A, None, A, 0) == INVALID
    assert status(api.attn_append_decode_planned_fp8, d, A, A, A, A, A, A, A, A, None, A, 0) == INVALID


def test_the_plan_calls_take_it():
    assert status(api.attn_plan, desc(), A, A, A, A, A, A, 0) not in (INVALID, UNSUPPORTED)
    assert status(api.attn_plan_append, desc(), A, A, A, A, A, A, A, A, 0) not in (INVALID, UNSUPPORTED)
    assert status(api.attn_plan_limited, desc(flags=api.HW_DESC_VIEW_LIMITS), A, A, A, A, A, A, A,
                  0) not in (INVALID, UNSUPPORTED)


@pytest.mark.parametrize("call,n", [("hw_attn_plan_tree", 11), ("hw_attn_decode_tree", 8), ("hw_tree_commit", 0)])
def test_draft_trees_refuse_the_description(call, n):
    f, d = getattr(api.lib(), call), ctypes.byref(desc())
    assert f(d, 4, *([A] * n if n else [1] + [A] * 5), 1 << 40, None) == INVALID


def test_no_rows_is_no_work():
    d = desc(n_rows=0)
    api.attn_decode_planned_fp4(d, None, None, None, None, None, None, None, 0)
    api.attn_append_decode_planned_fp4(d, None, None, None, None, None, None, None, None, None, 0)


def test_sessions():
    with pytest.raises(ValueError):  # one format
        engine.DecodeSession(n_rows=1, n_q_heads=4, n_kv_heads=2, head_dim=128, n_blocks=1, max_view_blocks=1, capacity=100,
                             dtype=torch.bfloat16, rope_theta=1e6, kv_fp8=True, kv_fp4=True)
