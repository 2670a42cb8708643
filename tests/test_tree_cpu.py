"""Host checks of the draft-tree calls: refusals before anything is enqueued."""
from __future__ import annotations

import ctypes

import pytest

from concurrent_shared_kv_gb300 import api

P = 1 << 20  # a non-null, aligned pointer that no refused call touches
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3


@pytest.fixture(scope="module")
def L():
    return api.lib()


def desc(**kw):
    a = dict(n_rows=2, n_q_heads=8, n_kv_heads=2, head_dim=128, n_blocks=3, max_view_blocks=3, cache_capacity=1000,
             dtype=api.HW_BF16, rope_theta=1e4, scale=0.1, flags=0)
    a.update(kw)
    return api.make_desc(**a)


def size(L, d, nodes):
    n = ctypes.c_size_t(0)
    return L.hw_attn_tree_workspace_size(ctypes.byref(d), nodes, ctypes.byref(n))


@pytest.mark.parametrize("kw,nodes,status", [
    ({}, 0, INVALID), ({}, -1, INVALID), ({}, 129, UNSUPPORTED), ({"flags": 1}, 4, UNSUPPORTED),
    ({"flags": 4}, 4, INVALID), ({"head_dim": 96}, 4, UNSUPPORTED), ({"dtype": 3}, 4, INVALID),
    ({"dtype": api.HW_FP8_E4M3, "head_dim": 64}, 4, UNSUPPORTED), ({"n_q_heads": 7}, 4, INVALID),
    ({"n_rows": 4097, "max_view_blocks": 0}, 1, UNSUPPORTED), ({"n_rows": 1024, "max_view_blocks": 1}, 65, UNSUPPORTED),
    ({"n_rows": -1}, 4, INVALID), ({"rope_theta": 1.0}, 4, INVALID)])
def test_descriptions(L, kw, nodes, status):
    assert size(L, desc(**kw), nodes) == status
    d = desc(**kw)
    assert L.hw_attn_plan_tree(ctypes.byref(d), nodes, *[P] * 11, 1 << 40, None) == status
    assert L.hw_tree_commit(ctypes.byref(d), nodes, 1, *[P] * 5, 1 << 40, None) == status
    if d.dtype != api.HW_FP8_E4M3:
        assert L.hw_attn_decode_tree(ctypes.byref(d), nodes, *[P] * 8, 1 << 40, None) == status


def test_no_rows_is_no_work(L):
    d = desc(n_rows=0)
    assert L.hw_attn_plan_tree(ctypes.byref(d), 4, *[None] * 11, 0, None) == OK
    assert L.hw_attn_decode_tree(ctypes.byref(d), 4, *[None] * 8, 0, None) == OK
    assert L.hw_tree_commit(ctypes.byref(d), 4, 3, *[None] * 5, 0, None) == OK
    assert L.hw_tree_commit(ctypes.byref(desc()), 4, 0, *[None] * 5, 0, None) == OK
    assert L.hw_tree_verify(0, 0, 4, 10, None, None, None, None, 10, None, 0, *[None] * 6) == OK


@pytest.mark.parametrize("missing", range(11))
def test_plan_arguments(L, missing):
    # block_start, block_len, view_block, view_offset, q_pos, q_to_kv, tree_block, tree_start, n_nodes, parent, workspace
    a = [P] * 11
    a[missing] = None
    want = WORKSPACE if missing in (5, 7, 10) else INVALID  # q_to_kv and tree_start may be NULL
    a[10] = None if missing in (5, 7) else a[10]            # (then the workspace is what is missing)
    assert L.hw_attn_plan_tree(ctypes.byref(desc()), 4, *a, 1 << 40, None) == want


@pytest.mark.parametrize("missing", range(8))
def test_decode_arguments(L, missing):
    # q, k_new, v_new, k_cache, v_cache, out, lse, workspace
    a = [P] * 8
    a[missing] = None
    a[7] = None if missing == 6 else a[7]
    want = WORKSPACE if missing >= 6 else INVALID  # lse may be NULL
    assert L.hw_attn_decode_tree(ctypes.byref(desc()), 4, *a, 1 << 40, None) == want


@pytest.mark.parametrize("odd", range(5))
def test_decode_alignment(L, odd):
    a = [P] * 8
    a[odd] = P + 8
    assert L.hw_attn_decode_tree(ctypes.byref(desc()), 4, *a, 1 << 40, None) == INVALID
    a = [P] * 8
    a[7] = P + 128  # the workspace at 256 bytes
    assert L.hw_attn_decode_tree(ctypes.byref(desc()), 4, *a, 1 << 40, None) == WORKSPACE


def test_types_have_their_calls(L):
    f8 = desc(dtype=api.HW_FP8_E4M3)
    assert L.hw_attn_decode_tree(ctypes.byref(f8), 4, *[P] * 8, 1 << 40, None) == UNSUPPORTED
    assert L.hw_attn_decode_tree_fp8(ctypes.byref(desc()), 4, *[P] * 10, 1 << 40, None) == INVALID
    for missing in (5, 6):  # the scales
        a = [P] * 10
        a[missing] = None
        assert L.hw_attn_decode_tree_fp8(ctypes.byref(f8), 4, *a, 1 << 40, None) == INVALID


@pytest.mark.parametrize("missing", range(5))
def test_commit_arguments(L, missing):
    a = [P] * 5  # k_cache, v_cache, path, n_path, workspace
    a[missing] = None
    assert L.hw_tree_commit(ctypes.byref(desc()), 4, 1, *a, 1 << 40, None) == (WORKSPACE if missing == 4 else INVALID)
    assert L.hw_tree_commit(ctypes.byref(desc()), 4, -1, *[P] * 5, 1 << 40, None) == INVALID
    a = [P + 8, P, P, P, P]
    assert L.hw_tree_commit(ctypes.byref(desc()), 4, 1, *a, 1 << 40, None) == INVALID


def verify(L, **kw):
    a = dict(dtype=0, n_rows=2, max_nodes=4, vocab=10, n_nodes=P, parent=P, token=P, p=P, p_stride=10, q=P, q_stride=10,
             u_accept=P, u_sample=P, path=P, n_path=P, next_token=P, stream=None)
    a.update(kw)
    return L.hw_tree_verify(*a.values())


@pytest.mark.parametrize("kw,status", [
    ({"dtype": 2}, INVALID), ({"dtype": 7}, INVALID), ({"n_rows": -1}, INVALID), ({"max_nodes": 0}, INVALID),
    ({"max_nodes": 129}, UNSUPPORTED), ({"vocab": 0}, INVALID), ({"p_stride": 9}, INVALID), ({"q_stride": 9}, INVALID),
    ({"vocab": (1 << 24) + 1, "p_stride": 1 << 25, "q_stride": 1 << 25}, UNSUPPORTED),
    ({"n_rows": 20000}, UNSUPPORTED), ({"p": P + 2}, INVALID), ({"q": P + 1, "dtype": 1}, INVALID),
    ({"n_nodes": None}, INVALID), ({"parent": None}, INVALID), ({"token": None}, INVALID), ({"p": None}, INVALID),
    ({"u_accept": None}, INVALID), ({"u_sample": None}, INVALID), ({"path": None}, INVALID),
    ({"n_path": None}, INVALID), ({"next_token": None}, INVALID)])
def test_verify_arguments(L, kw, status):
    assert verify(L, **kw) == status


def test_verify_tensor_layouts():
    torch = pytest.importorskip("torch")
    from concurrent_shared_kv_gb300 import engine
    i = torch.zeros(2, 3, dtype=torch.int32)
    u = torch.zeros(2, 3)
    p = torch.zeros(2, 3, 8)
    with pytest.raises(ValueError):
        engine.tree_verify(i[:, 0], i, i, p, p[..., :7], u, u[:, 0])
    with pytest.raises(ValueError):
        engine.tree_verify(i[:, 0], i, i, p, p.bfloat16(), u, u[:, 0])
    with pytest.raises(ValueError):
        engine.tree_verify(i[:, 0], i, i, p[..., ::2], None, u, u[:, 0])
    with pytest.raises(ValueError):
        engine.tree_verify(i[:, 0], i, i, torch.zeros(4, 3, 8)[::2], None, u, u[:, 0])


def test_tensors_that_do_not_fit_are_refused():
    """What a kernel would read past: refused before the library is called."""
    torch = pytest.importorskip("torch")
    from concurrent_shared_kv_gb300 import engine
    i, f, p = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3), torch.zeros(2, 3, 8)
    good = dict(n_nodes=i[:, 0].contiguous(), parent=i, token=i, p=p, q=None, u_accept=f, u_sample=f[:, 0].contiguous())
    for name, bad in (("n_nodes", i[0]), ("n_nodes", i[:, 0]), ("parent", i[:, :2]), ("parent", i.long()), ("token", i[:1]),
                      ("u_accept", f.double()), ("u_accept", f[:, :2]), ("u_sample", f[0])):
        with pytest.raises(ValueError, match=name):
            engine.tree_verify(**{**good, name: bad})
    s = object.__new__(engine.TreeSession)   # (a session needs a device)
    s.desc, s.max_nodes, s.device = desc(n_rows=2, max_view_blocks=2), 3, torch.device("cpu")
    s.dtype = s.cache_dtype = torch.bfloat16
    s.sizes, s.workspace, s.ws_bytes = (2 * 3 * 8 * 128, 2 * 3 * 2 * 128, 2 * 1000 * 128), None, 0
    meta = dict(block_start=[0] * 3, block_len=[0] * 3, view_block=[[0, 1]] * 2, view_offset=[[0, 1]] * 2, q_pos=[0, 0])
    for name, bad in (("block_start", [0, 1]), ("view_block", [[0]] * 2), ("view_offset", [0] * 3), ("q_pos", [0])):
        with pytest.raises(ValueError, match=name):
            s.set_metadata(**{**meta, name: bad})
    with pytest.raises(ValueError, match="q_to_kv"):
        s.set_metadata(**meta, q_to_kv=[0])
    s.set_metadata(**meta)
    trees = dict(tree_block=[0, 1], n_nodes=[1, 1], parent=[[-1] * 3] * 2, tree_start=[0, 5])
    for name, bad in (("tree_block", [0]), ("n_nodes", [1]), ("parent", [[-1] * 2] * 2), ("tree_start", [0])):
        with pytest.raises(ValueError, match=name):
            s.plan(**{**trees, name: bad})
    bf = dict(dtype=torch.bfloat16)
    layer = dict(q=torch.zeros(2, 3, 8, 128, **bf), k_new=torch.zeros(2, 3, 2, 128, **bf), v_new=torch.zeros(2, 3, 2, 128, **bf),
                 k_cache=torch.zeros(2, 1000, 128, **bf), v_cache=torch.zeros(2, 1000, 128, **bf),
                 out=torch.zeros(2, 3, 8, 128, **bf), lse=torch.zeros(2, 3, 8))
    for name, bad in (("q", layer["q"][:, :2]), ("q", layer["q"].float()), ("q", layer["q"].transpose(1, 2)),
                      ("k_new", layer["k_new"][:1]), ("v_new", layer["q"]), ("k_cache", layer["k_cache"][:, :999]),
                      ("v_cache", layer["v_cache"].float()), ("out", layer["q"][:1]), ("lse", torch.zeros(2, 3, 7))):
        with pytest.raises(ValueError, match=name):
            s.decode(**{**layer, name: bad})
    step = dict(k_cache=layer["k_cache"], v_cache=layer["v_cache"], path=i, n_path=i[:, 0].contiguous())
    for name, bad in (("k_cache", layer["k_cache"][:1]), ("v_cache", layer["v_cache"][:, 1:]), ("path", i[:, :2]), ("n_path", i)):
        with pytest.raises(ValueError, match=name):
            s.commit(**{**step, name: bad})


def cpu_session(engine, torch):
    """A session without a device: what it checks before the library is called."""
    s = object.__new__(engine.TreeSession)
    s.desc, s.max_nodes, s.device = desc(n_rows=2, max_view_blocks=2), 3, torch.device("cpu")
    s.dtype = s.cache_dtype = torch.bfloat16
    s.sizes, s.workspace, s.ws_bytes, s.meta = (2 * 3 * 8 * 128, 2 * 3 * 2 * 128, 2 * 1000 * 128), None, 0, None
    return s


def test_refused_tensors_do_not_stay(monkeypatch):
    """After a refusal the session holds what it held before."""
    torch = pytest.importorskip("torch")
    from concurrent_shared_kv_gb300 import engine
    s = cpu_session(engine, torch)
    calls = []
    monkeypatch.setattr(engine.api, "attn_plan_tree", lambda *a, **kw: calls.append((a, kw)))
    meta = dict(block_start=[0] * 3, block_len=[1] * 3, view_block=[[0, 1]] * 2, view_offset=[[0, 1]] * 2, q_pos=[0, 0])
    trees = dict(tree_block=[0, 1], n_nodes=[1, 1], parent=[[-1] * 3] * 2)
    with pytest.raises(ValueError):
        s.plan(**trees)                      # no views yet
    with pytest.raises(ValueError, match="q_pos"):
        s.set_metadata(**{**meta, "q_pos": [0]})
    with pytest.raises(ValueError):
        s.plan(**trees)                      # still none
    s.set_metadata(**meta)
    for bad in (dict(meta, block_len=[7]), dict(meta, view_block=[[7]] * 2), dict(meta, q_to_kv=[0])):
        with pytest.raises(ValueError):
            s.set_metadata(**bad)
    s.plan(**trees)
    with pytest.raises(ValueError):
        s.plan(**{**trees, "parent": [[-1] * 2] * 2})
    assert len(calls) == 1 and s.trees[2].numel() == 6
    a, kw = calls[0]
    assert [x.numel() for x in a[2:7]] == [3, 3, 4, 4, 2] and a[3].tolist() == [1] * 3 and kw["q_to_kv"] is None


def test_tensors_of_another_device_are_refused(monkeypatch):
    """A kernel would be handed an address that is not its own: refused, as are
    tensors that are on no GPU at all."""
    torch = pytest.importorskip("torch")
    from concurrent_shared_kv_gb300 import engine

    def called(*a, **kw):
        raise AssertionError("the library was called")
    for name in ("attn_plan_tree", "attn_decode_tree", "attn_decode_tree_fp8", "tree_commit", "tree_verify"):
        monkeypatch.setattr(engine.api, name, called)
    i, f, p = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3), torch.zeros(2, 3, 8)
    good = dict(n_nodes=i[:, 0].contiguous(), parent=i, token=i, p=p, q=p, u_accept=f, u_sample=f[:, 0].contiguous(), path=i.clone(),
                n_path=i[:, 0].contiguous(), next_token=i[:, 0].contiguous())
    for name in good:
        if name != "p":
            with pytest.raises(ValueError, match=f"{name} is on the device meta"):
                engine.tree_verify(**{**good, name: good[name].to("meta")})
    with pytest.raises(ValueError, match="on a GPU"):
        engine.tree_verify(**good)
    s = cpu_session(engine, torch)
    bf = dict(dtype=torch.bfloat16)
    layer = dict(q=torch.zeros(2, 3, 8, 128, **bf), k_new=torch.zeros(2, 3, 2, 128, **bf), v_new=torch.zeros(2, 3, 2, 128, **bf),
                 k_cache=torch.zeros(2, 1000, 128, **bf), v_cache=torch.zeros(2, 1000, 128, **bf),
                 out=torch.zeros(2, 3, 8, 128, **bf), lse=torch.zeros(2, 3, 8))
    scales = dict(k_scale=torch.ones(2), v_scale=torch.ones(2))
    for name in layer:
        with pytest.raises(ValueError, match=f"{name} is on the device meta"):
            s.decode(**{**layer, name: layer[name].to("meta")})
    step = dict(k_cache=layer["k_cache"], v_cache=layer["v_cache"], path=i, n_path=i[:, 0].contiguous())
    for name in step:
        with pytest.raises(ValueError, match=f"{name} is on the device meta"):
            s.commit(**{**step, name: step[name].to("meta")})
    for name in scales:
        with pytest.raises(ValueError, match=f"{name} is on the device meta"):
            s.decode_fp8(**layer, **{**scales, name: scales[name].to("meta")})
    # a GPU that is not the current one
    monkeypatch.setattr(engine.api, "current_device", lambda: 1)
    s.device = torch.device("cuda", 0)
    monkeypatch.setattr(engine, "_fits", lambda *a: None)
    monkeypatch.setattr(engine, "_pool_fits", lambda *a: None)
    monkeypatch.setattr(engine, "_int32", lambda x, *a: x)
    s.set_metadata([], [], [], [], [])
    for call in (lambda: s.decode(**layer), lambda: s.commit(**step), lambda: s.plan([], [], [])):
        with pytest.raises(ValueError, match="not the current device"):
            call()
    with pytest.raises(ValueError, match="on a GPU"):
        engine.TreeSession(n_rows=1, max_nodes=1, n_q_heads=1, n_kv_heads=1, head_dim=64, n_blocks=1, max_view_blocks=1, capacity=8,
                           dtype=torch.float32, rope_theta=1e4, device="cpu")


@pytest.mark.parametrize("cache,good,bad", [
    ("bfloat16", ["bfloat16"], ["float16", "int16", "float32", "uint8"]), ("float32", ["float32"], ["int32", "bfloat16", "float64"]),
    ("float8_e4m3fn", ["float8_e4m3fn", "uint8"], ["float8_e5m2", "int8", "bfloat16"])])
def test_pools_of_another_type_are_refused(monkeypatch, cache, good, bad):
    """A type of the same size is read as something else."""
    torch = pytest.importorskip("torch")
    from concurrent_shared_kv_gb300 import engine
    s = cpu_session(engine, torch)
    s.cache_dtype = getattr(torch, cache)
    s.dtype = torch.float32 if cache == "float32" else torch.bfloat16
    calls = []
    for name in ("attn_decode_tree", "attn_decode_tree_fp8", "tree_commit"):
        monkeypatch.setattr(engine.api, name, lambda *a, **kw: calls.append(a))

    def new(dtype, *shape):
        return torch.zeros(*shape).to(dtype)
    q, kn = new(s.dtype, 2, 3, 8, 128), new(s.dtype, 2, 3, 2, 128)
    path, n_path = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    ok = new(s.cache_dtype, 2, 1000, 128)
    for names, refused in ((good, False), (bad, True)):
        for name in names:
            x = new(getattr(torch, name), 2, 1000, 128)
            for k, v, what in ((x, ok, "k_cache"), (ok, x, "v_cache")):
                for call in (lambda: s.decode(q, kn, kn, k, v, out=q, want_lse=False), lambda: s.commit(k, v, path, n_path),
                             lambda: s.decode_fp8(q, kn, kn, k, v, torch.ones(2), torch.ones(2), out=q, want_lse=False)):
                    if refused:
                        with pytest.raises(ValueError, match=what):
                            call()
                    else:
                        call()
    assert len(calls) == 6 * len(good)


def test_a_call_makes_its_tensors_on_its_stream(monkeypatch):
    """Conversions, uploads and outputs of a call with stream= belong to that
    stream, those of a call without one to the current stream."""
    torch = pytest.importorskip("torch")
    import contextlib
    from concurrent_shared_kv_gb300 import engine
    now, made = [None], []

    @contextlib.contextmanager
    def on(stream):
        before, now[0] = now[0], stream
        yield
        now[0] = before
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: handle, raising=False)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    for module, name in ((engine, "_int32"), (torch, "empty")):
        real = getattr(module, name)
        monkeypatch.setattr(module, name, lambda *a, real=real, **kw: (made.append(now[0]), real(*a, **kw))[1])
    for name in ("attn_plan_tree", "attn_decode_tree", "attn_decode_tree_fp8", "tree_verify"):
        monkeypatch.setattr(engine.api, name, lambda *a, **kw: None)
    monkeypatch.setattr(engine, "_on_gpu", lambda device: None)

    class Handle:  # another library's stream
        cuda_stream = 99

    s = cpu_session(engine, torch)
    bf = dict(dtype=torch.bfloat16)
    q, kn, k = torch.zeros(2, 3, 8, 128, **bf), torch.zeros(2, 3, 2, 128, **bf), torch.zeros(2, 1000, 128, **bf)
    i, f, p = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3), torch.zeros(2, 3, 8)
    for stream, want in ((None, None), (77, 77), (0, "default"), (Handle(), 99)):
        made.clear()
        s.set_metadata([0] * 3, [1] * 3, [[0, 1]] * 2, [[0, 1]] * 2, [0, 0], q_to_kv=[0] * 8, stream=stream)
        s.plan([0, 1], torch.tensor([1, 1]), [[-1] * 3] * 2, tree_start=[0, 5], stream=stream)
        assert len(made) == 10
        s.decode(q, kn, kn, k, k, stream=stream)
        s.decode_fp8(q, kn, kn, k, k, torch.ones(2), torch.ones(2), stream=stream)
        engine.tree_verify(i[:, 0].contiguous(), i, i, p, None, f, f[:, 0].contiguous(), stream=stream)
        assert made == [want] * 17
        s.decode(q, kn, kn, k, k, out=q, want_lse=False, stream=stream)
        assert len(made) == 17 and now[0] is None
