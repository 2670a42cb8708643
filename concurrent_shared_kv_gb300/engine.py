"""Torch-facing convenience layer over the C ABI: it owns a workspace and the
device copies of the per-step metadata.  PyTorch only allocates memory and
provides streams here; every step of the computation runs in libhogwild."""
from __future__ import annotations

import contextlib
from typing import Optional

import numpy as np
import torch

from . import api

DTYPES = {torch.float32: api.HW_F32, torch.bfloat16: api.HW_BF16,
          torch.uint8: api.HW_FP8_E4M3, torch.float8_e4m3fn: api.HW_FP8_E4M3}


class DecodeSession:
    """One decode configuration: shapes, pools, workspace and metadata."""

    def __init__(self, *, n_rows: int, n_q_heads: int, n_kv_heads: int, head_dim: int,
                 n_blocks: int, max_view_blocks: int, capacity: int, dtype: torch.dtype,
                 rope_theta: float, scale: Optional[float] = None, device="cuda",
                 view_limits: bool = False, kv_fp8: bool = False, kv_fp4: bool = False):
        """view_limits: the steps are planned with per-view-entry token limits
        (plan_limited; decode_planned then applies them).  kv_fp8: the K and V
        pools hold E4M3 codes with per-kv-head scales (decode_planned_fp8);
        kv_fp4: E2M1 codes with a scale a token (decode_planned_fp4); dtype is
        then that of q and out (bf16)."""
        if kv_fp4 and (kv_fp8 or dtype != torch.bfloat16):
            raise ValueError("4-bit caches: dtype bfloat16, and not kv_fp8")
        self.device = torch.device(device)
        self.dtype = dtype
        storage = api.HW_FP4_E2M1 if kv_fp4 else api.HW_FP8_E4M3 if kv_fp8 else DTYPES[dtype]
        self.desc = api.make_desc(n_rows, n_q_heads, n_kv_heads, head_dim, n_blocks,
                                  max_view_blocks, capacity,
                                  storage, rope_theta,
                                  head_dim ** -0.5 if scale is None else scale,
                                  flags=api.HW_DESC_VIEW_LIMITS if view_limits else 0)
        # the same description with the early-loads promise (see early= below)
        self.desc_early = api.make_desc(n_rows, n_q_heads, n_kv_heads, head_dim, n_blocks,
                                        max_view_blocks, capacity,
                                        storage, rope_theta,
                                        head_dim ** -0.5 if scale is None else scale,
                                        flags=self.desc.flags | api.HW_DESC_EARLY_LOADS)
        self.ws_bytes = api.attn_decode_workspace_size(self.desc)
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
        api.workspace_init(self.workspace, self.ws_bytes)
        self.meta = None

    def set_metadata(self, block_start, block_len, view_block, view_offset, q_pos, q_to_kv=None,
                     non_blocking: bool = False):
        """Upload the step's metadata (shared by every layer of the step)."""
        def dev(x):
            if x is None:
                return None
            t = torch.as_tensor(np.ascontiguousarray(x, dtype=np.int32)) if not torch.is_tensor(x) else x
            return t.to(self.device, dtype=torch.int32, non_blocking=non_blocking).contiguous()
        self.meta = dict(block_start=dev(block_start), block_len=dev(block_len),
                         view_block=dev(view_block), view_offset=dev(view_offset),
                         q_pos=dev(q_pos), q_to_kv=dev(q_to_kv))

    def decode(self, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
               out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
               want_lse: bool = True, stream=None, early: bool = False):
        d = self.desc_early if early else self.desc
        if out is None:
            out = torch.empty((d.n_rows, d.n_q_heads, d.head_dim), dtype=self.dtype, device=self.device)
        if lse is None and want_lse:
            lse = torch.empty((d.n_rows, d.n_q_heads), dtype=torch.float32, device=self.device)
        m = self.meta
        api.attn_decode(d, q, k_cache, v_cache, m["block_start"], m["block_len"], m["view_block"],
                        m["view_offset"], m["q_pos"], out, lse, self.workspace, self.ws_bytes,
                        q_to_kv=m["q_to_kv"], stream=stream)
        return out, lse

    def plan(self, stream=None):
        """hw_attn_plan on the uploaded metadata: once per step, before the
        layers' decode_planned calls."""
        m = self.meta
        api.attn_plan(self.desc, m["block_start"], m["block_len"], m["view_block"],
                      m["view_offset"], m["q_pos"], self.workspace, self.ws_bytes,
                      q_to_kv=m["q_to_kv"], stream=stream)

    def plan_limited(self, view_limit, stream=None):
        """hw_attn_plan_limited: plan the step with a token limit per view
        entry ([rows][V]; negative = the whole block), e.g. the causal order
        of a chunk of queries within its own block."""
        m = self.meta
        t = torch.as_tensor(np.ascontiguousarray(view_limit, dtype=np.int32)) \
            if not torch.is_tensor(view_limit) else view_limit
        self.view_limit = t.to(self.device, dtype=torch.int32).contiguous()
        api.attn_plan_limited(self.desc, m["block_start"], m["block_len"], m["view_block"],
                              m["view_offset"], self.view_limit, m["q_pos"], self.workspace,
                              self.ws_bytes, q_to_kv=m["q_to_kv"], stream=stream)

    def plan_append(self, append_block, append_pos, stream=None):
        """hw_attn_plan_append: plan the step with each row's new token
        (append_block[r] = its block or -1, append_pos[r] = its block-local
        position; block_len of the uploaded metadata must count it)."""
        m = self.meta
        def dev(x):
            t = torch.as_tensor(np.ascontiguousarray(x, dtype=np.int32)) if not torch.is_tensor(x) else x
            return t.to(self.device, dtype=torch.int32).contiguous()
        self.append = (dev(append_block), dev(append_pos))
        api.attn_plan_append(self.desc, m["block_start"], m["block_len"], m["view_block"],
                             m["view_offset"], m["q_pos"], self.append[0], self.append[1],
                             self.workspace, self.ws_bytes, q_to_kv=m["q_to_kv"], stream=stream)

    def append_decode_planned(self, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                              k_cache: torch.Tensor, v_cache: torch.Tensor,
                              out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                              want_lse: bool = True, stream=None, early: bool = False):
        """One layer: its new tokens ([rows][Hkv][D]) written, then decoded."""
        d = self.desc_early if early else self.desc
        if out is None:
            out = torch.empty((d.n_rows, d.n_q_heads, d.head_dim), dtype=self.dtype, device=self.device)
        if lse is None and want_lse:
            lse = torch.empty((d.n_rows, d.n_q_heads), dtype=torch.float32, device=self.device)
        api.attn_append_decode_planned(d, q, k_new, v_new, k_cache, v_cache, out, lse,
                                       self.workspace, self.ws_bytes, stream=stream)
        return out, lse

    def decode_planned(self, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                       out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                       want_lse: bool = True, stream=None, early: bool = False):
        """One layer against the step's plan (see plan()).  early=True promises
        that the work enqueued just before this call on the stream writes
        neither this layer's K/V pools nor the plan (HW_DESC_EARLY_LOADS): true
        for every layer of a step after the first one that follows the plan."""
        d = self.desc_early if early else self.desc
        if out is None:
            out = torch.empty((d.n_rows, d.n_q_heads, d.head_dim), dtype=self.dtype, device=self.device)
        if lse is None and want_lse:
            lse = torch.empty((d.n_rows, d.n_q_heads), dtype=torch.float32, device=self.device)
        api.attn_decode_planned(d, q, k_cache, v_cache, out, lse, self.workspace, self.ws_bytes,
                                stream=stream)
        return out, lse

    def decode_planned_fp8(self, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                           k_scale: torch.Tensor, v_scale: torch.Tensor,
                           out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                           want_lse: bool = True, stream=None, early: bool = False):
        """One layer over E4M3 pools (codes, [Hkv][cap][D]) with float32 scales [Hkv]."""
        d = self.desc_early if early else self.desc
        if out is None:
            out = torch.empty((d.n_rows, d.n_q_heads, d.head_dim), dtype=self.dtype, device=self.device)
        if lse is None and want_lse:
            lse = torch.empty((d.n_rows, d.n_q_heads), dtype=torch.float32, device=self.device)
        api.attn_decode_planned_fp8(d, q, k_cache, v_cache, k_scale, v_scale, out, lse,
                                    self.workspace, self.ws_bytes, stream=stream)
        return out, lse

    def append_decode_planned_fp8(self, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                                  k_cache: torch.Tensor, v_cache: torch.Tensor,
                                  k_scale: torch.Tensor, v_scale: torch.Tensor,
                                  out: Optional[torch.Tensor] = None,
                                  lse: Optional[torch.Tensor] = None, want_lse: bool = True,
                                  stream=None, early: bool = False):
        """One layer over E4M3 pools: its new tokens (bf16, [rows][Hkv][D])
        written as codes with the head scales, then decoded."""
        d = self.desc_early if early else self.desc
        if out is None:
            out = torch.empty((d.n_rows, d.n_q_heads, d.head_dim), dtype=self.dtype, device=self.device)
        if lse is None and want_lse:
            lse = torch.empty((d.n_rows, d.n_q_heads), dtype=torch.float32, device=self.device)
        api.attn_append_decode_planned_fp8(d, q, k_new, v_new, k_cache, v_cache, k_scale, v_scale,
                                           out, lse, self.workspace, self.ws_bytes, stream=stream)
        return out, lse

    def _fp4_layer(self, q, k_cache, v_cache, kv_scale, out, lse, want_lse, stream, new=()):
        """The outputs of a layer over 4-bit caches, and what a kernel would
        read past checked."""
        d, dev = self.desc, q.device
        if d.dtype != api.HW_FP4_E2M1:
            raise ValueError("the session has no 4-bit caches (kv_fp4)")
        n, rows = d.n_rows * d.n_q_heads, d.n_kv_heads * d.cache_capacity
        if out is None:
            out = _new((d.n_rows, d.n_q_heads, d.head_dim), self.dtype, dev, stream)
        if lse is None and want_lse:
            lse = _new((d.n_rows, d.n_q_heads), torch.float32, dev, stream)
        _fits("q", q, n * d.head_dim, self.dtype, self.workspace.device)
        _fits("out", out, n * d.head_dim, self.dtype, dev)
        if lse is not None:
            _fits("lse", lse, n, torch.float32, dev)
        _fits("k_cache", k_cache, rows * d.head_dim // 2, torch.uint8, dev)
        _fits("v_cache", v_cache, rows * d.head_dim // 2, torch.uint8, dev)
        _fits("kv_scale", kv_scale, rows * 2, torch.bfloat16, dev)
        for what, x in zip(("k_new", "v_new"), new):
            _fits(what, x, d.n_rows * d.n_kv_heads * d.head_dim, self.dtype, dev)
        _current(dev)
        return out, lse

    def decode_planned_fp4(self, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                           kv_scale: torch.Tensor, out: Optional[torch.Tensor] = None,
                           lse: Optional[torch.Tensor] = None, want_lse: bool = True, stream=None,
                           early: bool = False):
        """One layer over E2M1 pools (packed codes, uint8 [Hkv][cap][D / 2]) with
        the tokens' scales (bfloat16 [Hkv][cap][2]: key, value)."""
        out, lse = self._fp4_layer(q, k_cache, v_cache, kv_scale, out, lse, want_lse, stream)
        api.attn_decode_planned_fp4(self.desc_early if early else self.desc, q, k_cache, v_cache, kv_scale,
                                    out, lse, self.workspace, self.ws_bytes, stream=stream)
        return out, lse

    def append_decode_planned_fp4(self, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                                  k_cache: torch.Tensor, v_cache: torch.Tensor,
                                  kv_scale: torch.Tensor, out: Optional[torch.Tensor] = None,
                                  lse: Optional[torch.Tensor] = None, want_lse: bool = True,
                                  stream=None, early: bool = False):
        """One layer over E2M1 pools: its new tokens (bf16, [rows][Hkv][D])
        encoded into them, then decoded."""
        out, lse = self._fp4_layer(q, k_cache, v_cache, kv_scale, out, lse, want_lse, stream, (k_new, v_new))
        api.attn_append_decode_planned_fp4(self.desc_early if early else self.desc, q, k_new, v_new,
                                           k_cache, v_cache, kv_scale, out, lse, self.workspace,
                                           self.ws_bytes, stream=stream)
        return out, lse

    def device_flags(self) -> int:
        return api.workspace_status(self.workspace)


def _int32(x, device, stream=None):
    """x as dense int32 on the device, under _on(stream)."""
    t = torch.as_tensor(np.ascontiguousarray(x, dtype=np.int32)) if not torch.is_tensor(x) else x
    r = t.to(device, dtype=torch.int32).contiguous()
    if r is not t and t.is_cuda:
        _kept_for(stream, t)
    return r


def _on(stream, device):
    """The stream of a call as torch's current one: tensors made under it are
    made by it and go back to it."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):  # a handle
        handle = stream if isinstance(stream, int) else stream.cuda_stream
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _kept_for(stream, *tensors) -> None:
    """Memory that goes back to the stream it came from only once `stream` (None:
    the current one) is done with it.  (Not for handles: the allocator would
    have to use one that may be gone by then.)"""
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        for x in tensors:
            if x is not None and x.is_cuda:
                x.record_stream(stream)


def _new(shape, dtype, device, stream):
    """An output of a call on `stream`, for the caller's current one as well."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _on(stream, device):
        x = torch.empty(shape, dtype=dtype, device=device)
    if x.is_cuda:
        x.record_stream(torch.cuda.current_stream())
    return x


def _current(device) -> None:
    """Kernels are launched on the current device."""
    index = device.index  # (of a GPU)
    if index is not None and index != api.current_device():
        raise ValueError(f"{device} is not the current device")


def _on_gpu(device) -> None:
    if device.type != "cuda":
        raise ValueError(f"the calls need tensors on a GPU, not on {device}")
    _current(device)


def _misfit(what: str, x, n: int, dtype, device):
    if x.device != device:
        raise ValueError(f"{what} is on the device {x.device}, not on {device}")
    raise ValueError(f"{what} needs {n} dense elements of {dtype}, got {tuple(x.shape)} of {x.dtype}")


def _fits(what: str, x, n: int, dtype, device) -> None:
    """A dense tensor of n elements: what a kernel would read past otherwise."""
    if x.numel() != n or x.dtype != dtype or x.device != device or not x.is_contiguous():
        _misfit(what, x, n, dtype, device)


def _pool_fits(what: str, x, n: int, dtype, device) -> None:
    if x.numel() != n or x.device != device or not x.is_contiguous() or (
            x.dtype != dtype and (dtype != torch.float8_e4m3fn or x.dtype != torch.uint8)):  # (codes may be bytes)
        _misfit(what, x, n, dtype, device)


class TreeSession:
    """Steps whose rows each query a tree of drafted tokens: plan(), one
    decode() a layer, tree_verify(), commit().

    A call with stream= runs on that stream (a torch stream, or a handle), and
    what it makes - converted or uploaded arrays, outputs - is made there.  The
    caller's own tensors have to be there for that stream and stay until it has
    used them; a session whose calls have a handle is kept until they are done."""

    def __init__(self, *, n_rows: int, max_nodes: int, n_q_heads: int, n_kv_heads: int, head_dim: int,
                 n_blocks: int, max_view_blocks: int, capacity: int, dtype: torch.dtype,
                 rope_theta: float, scale: Optional[float] = None, device="cuda",
                 kv_fp8: bool = False):
        """max_nodes: nodes of the largest tree (q, out and the new tokens are
        [rows][max_nodes][heads][D]).  dtype, kv_fp8: as in DecodeSession."""
        self.device = torch.device(device)
        if self.device == torch.device("cuda"):
            self.device = torch.device("cuda", torch.cuda.current_device())
        _on_gpu(self.device)
        self.dtype = dtype
        self.max_nodes = int(max_nodes)
        self.desc = api.make_desc(n_rows, n_q_heads, n_kv_heads, head_dim, n_blocks,
                                  max_view_blocks, capacity,
                                  api.HW_FP8_E4M3 if kv_fp8 else DTYPES[dtype], rope_theta,
                                  head_dim ** -0.5 if scale is None else scale)
        self.ws_bytes = api.attn_tree_workspace_size(self.desc, self.max_nodes)
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
        api.workspace_init(self.workspace, self.ws_bytes)
        self.meta = None
        self.workspace_on = api._stream(None)  # the stream that its memory came from
        nodes = n_rows * self.max_nodes
        self.sizes = (nodes * n_q_heads * head_dim, nodes * n_kv_heads * head_dim, n_kv_heads * capacity * head_dim)
        self.cache_dtype = torch.float8_e4m3fn if kv_fp8 else dtype

    def set_metadata(self, block_start, block_len, view_block, view_offset, q_pos, q_to_kv=None, stream=None):
        """Upload the step's views: those of the rows' tokens before their trees.
        stream: the one that plan() will have."""
        with _on(stream, self.device):
            meta = [_int32(x, self.device, stream) for x in (block_start, block_len, view_block, view_offset, q_pos)]
            q_to_kv = None if q_to_kv is None else _int32(q_to_kv, self.device, stream)
        d = self.desc
        for what, x, n in zip(("block_start", "block_len", "view_block", "view_offset", "q_pos"), meta,
                              (d.n_blocks, d.n_blocks, d.n_rows * d.max_view_blocks, d.n_rows * d.max_view_blocks, d.n_rows)):
            _fits(what, x, n, torch.int32, self.device)
        if q_to_kv is not None:
            _fits("q_to_kv", q_to_kv, d.n_q_heads, torch.int32, self.device)
        self.meta, self.q_to_kv = meta, q_to_kv
        self.meta_on = api._stream(stream)

    def plan(self, tree_block, n_nodes, parent, tree_start=None, stream=None):
        """hw_attn_plan_tree: the step's trees (tree_start None: behind each row's block)."""
        if self.meta is None:
            raise ValueError("plan() needs the step's views: set_metadata() first")
        with _on(stream, self.device):
            trees = [_int32(x, self.device, stream) for x in (tree_block, n_nodes, parent)]
            tree_start = None if tree_start is None else _int32(tree_start, self.device, stream)
        R = self.desc.n_rows
        for what, x, n in zip(("tree_block", "n_nodes", "parent"), trees, (R, R, R * self.max_nodes)):
            _fits(what, x, n, torch.int32, self.device)
        if tree_start is not None:
            _fits("tree_start", tree_start, R, torch.int32, self.device)
        _current(self.device)
        self.trees, self.tree_start = trees, tree_start
        if self.device.type == "cuda" and not self.workspace_on == self.meta_on == api._stream(stream):
            _kept_for(stream, self.workspace, *self.meta, self.q_to_kv)
        api.attn_plan_tree(self.desc, self.max_nodes, *self.meta, *self.trees, self.workspace,
                           self.ws_bytes, tree_start=self.tree_start, q_to_kv=self.q_to_kv,
                           stream=stream)

    def _outputs(self, out, lse, want_lse, stream):
        d = self.desc
        shape = (d.n_rows, self.max_nodes, d.n_q_heads)
        if out is None:
            out = _new(shape + (d.head_dim,), self.dtype, self.device, stream)
        if lse is None and want_lse:
            lse = _new(shape, torch.float32, self.device, stream)
        return out, lse

    def _check_layer(self, q, k_new, v_new, k_cache, v_cache, out, lse):
        n_q, n_new, n_pool = self.sizes
        dtype, cache, dev = self.dtype, self.cache_dtype, self.device
        _fits("q", q, n_q, dtype, dev)
        _fits("k_new", k_new, n_new, dtype, dev)
        _fits("v_new", v_new, n_new, dtype, dev)
        _fits("out", out, n_q, dtype, dev)
        _pool_fits("k_cache", k_cache, n_pool, cache, dev)
        _pool_fits("v_cache", v_cache, n_pool, cache, dev)
        if lse is not None:
            _fits("lse", lse, n_q // self.desc.head_dim, torch.float32, dev)
        _current(dev)

    def decode(self, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
               k_cache: torch.Tensor, v_cache: torch.Tensor, out: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, want_lse: bool = True, stream=None):
        """One layer: the trees' tokens written into the cache, then attended.
        Rows of out and lse behind a tree's nodes keep what they hold."""
        out, lse = self._outputs(out, lse, want_lse, stream)
        self._check_layer(q, k_new, v_new, k_cache, v_cache, out, lse)
        api.attn_decode_tree(self.desc, self.max_nodes, q, k_new, v_new, k_cache, v_cache, out, lse,
                             self.workspace, self.ws_bytes, stream=stream)
        return out, lse

    def decode_fp8(self, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                   k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                   v_scale: torch.Tensor, out: Optional[torch.Tensor] = None,
                   lse: Optional[torch.Tensor] = None, want_lse: bool = True, stream=None):
        """decode() over E4M3 pools with float32 scales [Hkv]; q and the new tokens bf16."""
        out, lse = self._outputs(out, lse, want_lse, stream)
        self._check_layer(q, k_new, v_new, k_cache, v_cache, out, lse)
        _fits("k_scale", k_scale, self.desc.n_kv_heads, torch.float32, self.device)
        _fits("v_scale", v_scale, self.desc.n_kv_heads, torch.float32, self.device)
        api.attn_decode_tree_fp8(self.desc, self.max_nodes, q, k_new, v_new, k_cache, v_cache,
                                 k_scale, v_scale, out, lse, self.workspace, self.ws_bytes,
                                 stream=stream)
        return out, lse

    def commit(self, k_cache: torch.Tensor, v_cache: torch.Tensor, path: torch.Tensor,
               n_path: torch.Tensor, stream=None):
        """The accepted nodes (tree_verify's path and n_path) appended to the
        rows' blocks in every layer; pools [layers][Hkv][cap][D] or [Hkv][cap][D]."""
        layers = 1 if k_cache.dim() == 3 else k_cache.shape[0]
        n, R, cache, dev = layers * self.sizes[2], self.desc.n_rows, self.cache_dtype, self.device
        _pool_fits("k_cache", k_cache, n, cache, dev)
        _pool_fits("v_cache", v_cache, n, cache, dev)
        _fits("path", path, R * self.max_nodes, torch.int32, dev)
        _fits("n_path", n_path, R, torch.int32, dev)
        _current(dev)
        api.tree_commit(self.desc, self.max_nodes, layers, k_cache, v_cache, path, n_path,
                        self.workspace, self.ws_bytes, stream=stream)

    def device_flags(self) -> int:
        return api.workspace_status(self.workspace)


def tree_verify(n_nodes: torch.Tensor, parent: torch.Tensor, token: torch.Tensor, p: torch.Tensor,
                q: Optional[torch.Tensor], u_accept: torch.Tensor, u_sample: torch.Tensor,
                path: Optional[torch.Tensor] = None, n_path: Optional[torch.Tensor] = None,
                next_token: Optional[torch.Tensor] = None, stream=None):
    """hw_tree_verify: (path, n_path, next_token) of drafted trees.  p and q:
    [rows][max_nodes][vocab], float32 or bfloat16, the last dimension dense and
    the first two one stride apart; q None: the tokens were chosen, not drawn."""
    R, T, V = shape = p.shape

    def step(x):
        s0, s1, s2 = x.stride()
        if (s2 != 1 and V > 1) or (R > 1 and T > 1 and s0 != T * s1):
            raise ValueError("p and q need rows one stride apart with dense values")
        return s1 if T > 1 else s0 if R > 1 else V

    dev = p.device
    if q is not None:
        if q.shape != shape or q.dtype != p.dtype:
            raise ValueError("p and q differ in shape or type")
        if q.device != dev:
            _misfit("q", q, q.numel(), q.dtype, dev)
    i32 = torch.int32
    if path is None:
        path = _new((R, T), i32, dev, stream)
    if n_path is None:
        n_path = _new(R, i32, dev, stream)
    if next_token is None:
        next_token = _new(R, i32, dev, stream)
    _fits("n_nodes", n_nodes, R, i32, dev)
    _fits("parent", parent, R * T, i32, dev)
    _fits("token", token, R * T, i32, dev)
    _fits("path", path, R * T, i32, dev)
    _fits("n_path", n_path, R, i32, dev)
    _fits("next_token", next_token, R, i32, dev)
    _fits("u_accept", u_accept, R * T, torch.float32, dev)
    _fits("u_sample", u_sample, R, torch.float32, dev)
    if p.is_cuda:
        _current(dev)
    else:
        _on_gpu(dev)
    api.tree_verify(DTYPES[p.dtype], R, T, V, n_nodes, parent, token, p, step(p), q,
                    0 if q is None else step(q), u_accept, u_sample, path, n_path, next_token,
                    stream=stream)
    return path, n_path, next_token


def block_commit(k_src: torch.Tensor, v_src: torch.Tensor, src_begin: int, n_tokens: int,
                 k_dst: torch.Tensor, v_dst: torch.Tensor, dst_offset: int, pos_delta: int,
                 rope_theta: float, stream=None):
    """Pools shaped [layers][Hkv][cap][D] or [Hkv][cap][D]."""
    def dims(t):
        return (1,) + tuple(t.shape) if t.dim() == 3 else tuple(t.shape)
    L, H, cs, D = dims(k_src)
    _, _, cd, _ = dims(k_dst)
    return api.block_commit(DTYPES[k_src.dtype], L, H, D, rope_theta, k_src, v_src, cs, src_begin,
                            n_tokens, k_dst, v_dst, cd, dst_offset, pos_delta, stream=stream)


def block_commit_many(k_src: torch.Tensor, v_src: torch.Tensor, commits, k_dst: torch.Tensor,
                      v_dst: torch.Tensor, rope_theta: float, stream=None):
    """Several finished steps in one launch.  `commits`: (src_begin, n_tokens,
    dst_offset, pos_delta) tuples; pools as in block_commit."""
    def dims(t):
        return (1,) + tuple(t.shape) if t.dim() == 3 else tuple(t.shape)
    L, H, cs, D = dims(k_src)
    _, _, cd, _ = dims(k_dst)
    cols = list(zip(*commits)) if commits else [(), (), (), ()]
    return api.block_commit_many(DTYPES[k_src.dtype], L, H, D, rope_theta, k_src, v_src, cs, k_dst,
                                 v_dst, cd, *cols, stream=stream)


def _pools(k_cache, v_cache, kv_scale, what=""):
    """(dtype, layers, Hkv, capacity, D) of a cache's pools, [layers][Hkv][cap][D]
    or [Hkv][cap][D] (with kv_scale: packed codes, D / 2 bytes a token)."""
    shape, dtype, dev = k_cache.shape, k_cache.dtype, k_cache.device
    if len(shape) not in (3, 4):
        raise ValueError(f"pools are [layers][Hkv][cap][D] or [Hkv][cap][D], not {tuple(shape)}")
    heads, cap, width = shape[-3:]
    layers = shape[0] if len(shape) == 4 else 1
    if kv_scale is not None:
        if dtype != torch.uint8:
            raise ValueError("4-bit pools are bytes (torch.uint8)")
        _fits(f"kv_scale{what}", kv_scale, layers * heads * cap * 2, torch.bfloat16, dev)
    elif dtype not in DTYPES:
        raise ValueError(f"no cache of {dtype}")
    if not k_cache.is_contiguous():
        raise ValueError(f"k{what or '_cache'} is not dense")
    _fits(f"v{what or '_cache'}", v_cache, layers * heads * cap * width, dtype, dev)
    if dev.type == "cuda":
        _current(dev)
    else:
        _on_gpu(dev)
    return (DTYPES[dtype] if kv_scale is None else api.HW_FP4_E2M1, layers, heads, cap,
            width if kv_scale is None else 2 * width)


def _head_scales(dtype, k_scale, v_scale, n, device):
    if dtype == api.HW_FP8_E4M3:
        if k_scale is None or v_scale is None:
            raise ValueError("8-bit caches need k_scale and v_scale (4-bit ones: kv_scale)")
        _fits("k_scale", k_scale, n, torch.float32, device)
        _fits("v_scale", v_scale, n, torch.float32, device)


def cache_write(k_new: torch.Tensor, v_new: torch.Tensor, slot: torch.Tensor, pos: torch.Tensor,
                k_cache: torch.Tensor, v_cache: torch.Tensor, *, rope_theta: float,
                k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                kv_scale: Optional[torch.Tensor] = None, flags: Optional[torch.Tensor] = None,
                stream=None) -> None:
    """hw_cache_write: tokens k_new, v_new ([layers][n][Hkv][D], or without the
    layers) into the pools' tokens slot[n] (int32, -1: left out), keys rotated at
    pos[n] (int32).  E4M3 pools with k_scale, v_scale (float32 [layers][Hkv]), E2M1
    pools (uint8, D / 2 bytes a token) with kv_scale (bfloat16 [layers][Hkv][cap][2]).
    flags: int32 [1], HW_DEV_BAD_RANGE is ORed in for slots outside the pool."""
    dtype, layers, heads, cap, dim = _pools(k_cache, v_cache, kv_scale)
    dev, n = k_cache.device, slot.numel()
    act = torch.float32 if dtype == api.HW_F32 else torch.bfloat16
    _fits("slot", slot, n, torch.int32, dev)
    _fits("pos", pos, n, torch.int32, dev)
    _fits("k_new", k_new, layers * n * heads * dim, act, dev)
    _fits("v_new", v_new, layers * n * heads * dim, act, dev)
    _head_scales(dtype, k_scale, v_scale, layers * heads, dev)
    if flags is not None:
        _fits("flags", flags, 1, torch.int32, dev)
    api.cache_write(dtype, layers, n, heads, dim, rope_theta, k_new, v_new, slot, pos, k_cache, v_cache, k_scale,
                    v_scale, kv_scale, cap, flags, stream=stream)


def cache_read(slot: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, *,
               k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
               kv_scale: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
               v_out: Optional[torch.Tensor] = None, flags: Optional[torch.Tensor] = None, stream=None):
    """hw_cache_read: (k_out, v_out), the values of the pools' tokens slot[n],
    [layers][n][Hkv][D] (without the layers where the pools have none); the rows of
    tokens left out (-1) keep what they hold.  Pools and scales as in cache_write."""
    dtype, layers, heads, cap, dim = _pools(k_cache, v_cache, kv_scale)
    dev, n = k_cache.device, slot.numel()
    act = torch.float32 if dtype == api.HW_F32 else torch.bfloat16
    shape = ((layers,) if k_cache.dim() == 4 else ()) + (n, heads, dim)
    if k_out is None:
        k_out = _new(shape, act, dev, stream)
    if v_out is None:
        v_out = _new(shape, act, dev, stream)
    _fits("slot", slot, n, torch.int32, dev)
    _fits("k_out", k_out, layers * n * heads * dim, act, dev)
    _fits("v_out", v_out, layers * n * heads * dim, act, dev)
    _head_scales(dtype, k_scale, v_scale, layers * heads, dev)
    if flags is not None:
        _fits("flags", flags, 1, torch.int32, dev)
    api.cache_read(dtype, layers, n, heads, dim, k_cache, v_cache, k_scale, v_scale, kv_scale, cap, slot, k_out,
                   v_out, flags, stream=stream)
    return k_out, v_out


def block_commit_fp4(k_src: torch.Tensor, v_src: torch.Tensor, scale_src: torch.Tensor,
                     k_dst: torch.Tensor, v_dst: torch.Tensor, scale_dst: torch.Tensor, src_begin,
                     n_tokens, dst_offset, pos_delta, *, rope_theta: float, stream=None) -> None:
    """hw_block_commit_many_fp4: finished steps of 4-bit caches, one for each entry
    of the four host sequences; pools [layers][Hkv][cap][D / 2] (or without the
    layers), scales bfloat16 [layers][Hkv][cap][2]."""
    _, layers, heads, cs, dim = _pools(k_src, v_src, scale_src, "_src")
    _, ld, hd, cd, dd = _pools(k_dst, v_dst, scale_dst, "_dst")
    if (layers, heads, dim) != (ld, hd, dd) or k_src.device != k_dst.device:
        raise ValueError("the two caches differ in layers, heads, head_dim or device")
    api.block_commit_many_fp4(layers, heads, dim, rope_theta, k_src, v_src, scale_src, cs, k_dst, v_dst, scale_dst,
                              cd, src_begin, n_tokens, dst_offset, pos_delta, stream=stream)


def block_move(k_cache: torch.Tensor, v_cache: torch.Tensor, src_begin, n_tokens, dst_begin, *,
               kv_scale: Optional[torch.Tensor] = None, stream=None) -> None:
    """hw_block_move: token ranges of the pools moved one after the other (host
    sequences), in every layer; pools as in cache_write."""
    dtype, layers, heads, cap, dim = _pools(k_cache, v_cache, kv_scale)
    api.block_move(dtype, layers, heads, dim, k_cache, v_cache, kv_scale, cap, src_begin, n_tokens, dst_begin,
                   stream=stream)


def compact(k_cache: torch.Tensor, v_cache: torch.Tensor, block_start, block_len, *, room=None,
            kv_scale: Optional[torch.Tensor] = None, stream=None) -> np.ndarray:
    """The pools' blocks slid together over the tokens no block holds (room[b] tokens
    kept free behind block b): where each now starts."""
    new, src, n, dst = api.compact_moves(block_start, block_len, k_cache.shape[-2], room)
    block_move(k_cache, v_cache, src, n, dst, kv_scale=kv_scale, stream=stream)
    return new
