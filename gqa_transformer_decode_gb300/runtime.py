"""Torch-side convenience wrapper around the C ABI.

PyTorch only provides device memory and streams here: weights are uploaded as
int16 tensors holding the bf16 bit patterns, handed to ember_model_create (which
copies them into the library's own layout) and released.  Every forward step
runs in libember.so.
"""
from __future__ import annotations

import ctypes as C
import importlib.util
import typing

import numpy as np
import torch

from . import ember as E


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream_ptr(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream)


class Model:
    """One model on the current CUDA device."""

    def __init__(self, shape, weights: dict, max_tokens: int = 0, max_positions: int = 0,
                 device="cuda", weights_q8: int = 0):
        self.shape = shape
        self.device = torch.device(device)
        self.cfg = E.make_config(shape, max_tokens, max_positions, weights_q8)
        up = {}
        for name, a in weights.items():
            a = np.ascontiguousarray(a)
            assert a.dtype == np.uint16, name
            up[name] = torch.from_numpy(a.view(np.int16)).to(self.device)
        L = shape.layers
        self._lw = (E.ember_layer_weights * L)()
        for l in range(L):
            for f in E.LAYER_FIELDS:
                t = up.get(f"layers.{l}.{f}")
                setattr(self._lw[l], f, None if t is None else t.data_ptr())
        w = E.ember_weights()
        w.embed = up["embed"].data_ptr()
        w.final_norm = up["final_norm"].data_ptr()
        w.cls_w = up["cls_w"].data_ptr() if "cls_w" in up else None
        w.cls_b = up["cls_b"].data_ptr() if "cls_b" in up else None
        w.layers = self._lw
        torch.cuda.synchronize()
        self.handle = E.ember_model_create(self.cfg, w)
        del up
        self.V, self.H = shape.vocab, shape.hidden

    def close(self):
        if getattr(self, "handle", None):
            E.ember_model_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def kv_alloc(self, max_seqs: int, max_len: int) -> "KVCache":
        return KVCache(self, max_seqs, max_len)

    # -- calls (asynchronous on `stream`; check status with sync_status) ------
    def prefill(self, kv, seq, ids, start_pos, logits=None, argmax=None, hidden=None, stream=None):
        st = E.ember_prefill(self.handle, kv.handle, seq, _ptr(ids), ids.numel(), start_pos,
                             _ptr(logits), _ptr(argmax), _ptr(hidden), _stream_ptr(stream))
        E.check(st, "ember_prefill")

    def prefill_activations(self, kv, seq, ids, start_pos, acts, logits=None, argmax=None, stream=None):
        """Prefill that also writes the residual after every block at the last
        position into acts [layers, hidden] (f32 device tensor)."""
        st = E.ember_prefill_activations(self.handle, kv.handle, seq, _ptr(ids), ids.numel(), start_pos,
                                         _ptr(acts), _ptr(logits), _ptr(argmax), _stream_ptr(stream))
        E.check(st, "ember_prefill_activations")

    def decode_step(self, kv, seqs, ids, positions, logits=None, argmax=None, stream=None):
        st = E.ember_decode_step(self.handle, kv.handle, ids.numel(), _ptr(seqs), _ptr(ids),
                                 _ptr(positions), _ptr(logits), _ptr(argmax), _stream_ptr(stream))

        E.check(st, "ember_decode_step")

    def decode_step_traced(self, kv, seqs, ids, positions, logits=None, argmax=None, stream=None):
        """The same step run eagerly, one kernel at a time, each launch timed
        with CUDA events: [(kernel name, device us)] in launch order."""
        st, tr = E.ember_decode_step_traced(self.handle, kv.handle, ids.numel(), _ptr(seqs), _ptr(ids),
                                            _ptr(positions), _ptr(logits), _ptr(argmax),
                                            _stream_ptr(stream))
        E.check(st, "ember_decode_step_traced")
        return [(E.kernel_name(n), us) for n, us in tr]

    def encode(self, ids, B, T, out=None, hidden=None, stream=None):
        st = E.ember_encode(self.handle, _ptr(ids), B, T, _ptr(out), _ptr(hidden),
                            _stream_ptr(stream))
        E.check(st, "ember_encode")

    def sync_status(self, stream=None) -> int:
        return E.ember_sync_status(self.handle, _stream_ptr(stream))


class KVCache:
    def __init__(self, model: Model, max_seqs: int, max_len: int):
        self.model = model
        self.max_seqs, self.max_len = max_seqs, max_len
        self.handle = E.ember_kv_alloc(model.handle, max_seqs, max_len)

    def reset(self, seq, stream=None):
        E.ember_kv_reset(self.handle, seq, _stream_ptr(stream))

    def set_cursor(self, seq, pos, stream=None):
        E.ember_kv_set_cursor(self.handle, seq, pos, _stream_ptr(stream))

    def tensors(self):
        """(K, V) int16 tensors [S, L, NKV, max_len, D] aliasing the cache (read only)."""
        k, v, strides = E.ember_kv_layout(self.handle)
        s = self.model.shape
        shape = (self.max_seqs, s.layers, s.n_kv_heads, self.max_len, s.head_dim)
        n = int(np.prod(shape))
        out = []
        for p in (k, v):
            buf = _wrap_device(p, n * 2, self.model.device)
            out.append(buf.view(torch.int16).view(shape))
        return tuple(out)

    def close(self):
        if getattr(self, "handle", None):
            E.ember_kv_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class PagedKV:
    """The paged K/V cache operators on torch tensors (include/ember.h, "paged
    key/value cache"): append new tokens' rows, attend with one token per
    sequence (decode) or several (prefill).

    k_pages, v_pages  bf16 or f16 [n_pages, n_kv_heads, page_size, head_dim]; any
                      strides with head_dim contiguous, the same for both, so
                      memory may also hold a row's heads side by side (a
                      transposed view)
    table             int32 [n_seqs, table_width], the sequences' pages

    The tensors stay the caller's and may change between calls, and be moved to
    other storage of the same type, shape, strides and device (t.data = ..); the object
    keeps references and one int32 status word.  Calls are asynchronous on
    `stream` (default: the current stream of the pages' device); device-side
    errors are read with sync_status().  A stream that is passed does not wait
    for the current one: the caller orders it after whatever made the inputs
    (wait_stream); the call keeps their memory, freed or not, until the stream is
    done with it.  (A stream made current instead has torch's own rules:
    record_stream is the caller's.)  Tensors that a call allocates are allocated
    on the call's stream, and hold anything in the rows that the call does not
    write (padding, rows outside every sequence).  The operators have no
    gradient: a tensor that requires one, the pages among them, is refused unless
    gradients are off, and so is one with a forward-mode tangent.
    """

    def __init__(self, k_pages, v_pages, table):
        if k_pages.dim() != 4 or k_pages.shape != v_pages.shape:
            raise ValueError("k_pages and v_pages must be alike: [n_pages, n_kv_heads, page_size, head_dim]")
        if k_pages.dtype not in _PAGE_DTYPES or v_pages.dtype != k_pages.dtype:
            raise TypeError("pages must be bfloat16 or float16")
        if table.dim() != 2 or table.dtype != torch.int32 or not table.is_contiguous():
            raise ValueError("table must be contiguous int32 [n_seqs, table_width]")
        if not k_pages.is_cuda or v_pages.device != k_pages.device or table.device != k_pages.device:
            raise ValueError("pages and table must be on one CUDA device")
        # the stride of a dimension of one is never walked: any valid value will do
        strides = [[t.stride(i) if t.shape[i] > 1 else t.shape[3] for i in range(3)] for t in (k_pages, v_pages)]
        if strides[0] != strides[1] or k_pages.stride(3) != 1 or v_pages.stride(3) != 1:
            raise ValueError("pages must have the same strides and head_dim contiguous")
        self.k_pages, self.v_pages, self.table = k_pages, v_pages, table
        self.device, self.dtype = k_pages.device, k_pages.dtype
        n_pages, self.n_kv_heads, page_size, self.head_dim = k_pages.shape
        c = E.ember_paged_kv()
        c.k, c.v, c.table = k_pages.data_ptr(), v_pages.data_ptr(), table.data_ptr()
        c.dtype = _PAGE_DTYPES[k_pages.dtype]
        c.n_pages, c.page_size, c.n_kv_heads, c.head_dim = n_pages, page_size, self.n_kv_heads, self.head_dim
        c.n_seqs, c.table_width = table.shape
        c.page_stride, c.head_stride, c.row_stride = strides[0]
        self.status = _status_word(self.device)
        self._t = _paged_torch()
        self._cache = self._t.cache(C.addressof(c), self.status.data_ptr(), k_pages.get_device(), k_pages, v_pages,
                                    self.status, table)

    def _on(self, stream):
        if stream.device != self.device:
            raise ValueError(f"the stream belongs to {stream.device}, the cache to {self.device}")
        return torch.cuda.stream(stream)

    def _call(self, stream, f, *args):
        """f on another stream: what it reads and writes stays allocated until it has run there."""
        with self._on(stream):
            r = f(*args)
        _keep_for(stream, *args, self.k_pages, self.v_pages, self.table)
        return r

    # -- operators ------------------------------------------------------------
    def append(self, k, v, seqs, positions, cos, sin, q=None, q_norm=None, k_norm=None, eps=1e-6, q_out=None,
               stream=None):
        """Norm (optional), rotate and store the K/V rows of new tokens.

        k, v [n, n_kv_heads, head_dim] and q [n, n_heads, head_dim] (optional) of
        one type, f32, bf16 or f16; seqs, positions int32 [n]; cos, sin f32
        [n_pos, head_dim / 2]; q_norm, k_norm bf16 [head_dim].  Returns the
        rotated queries in the cache's type (q_out where given), or None."""
        if stream is not None:
            return self._call(stream, self.append, k, v, seqs, positions, cos, sin, q, q_norm, k_norm, eps, q_out)
        return self._t.append(self._cache, k, v, seqs, positions, cos, sin, q, q_norm, k_norm, eps, q_out)

    def decode(self, q, lens, seqs=None, window=0, sinks=0, scale=None, out=None, lse=None, return_lse=False,
               workspace=None, stream=None):
        """Attention of one token per sequence: q [B, n_heads, head_dim], lens
        int32 [B] (keys of each sequence, the token's own among them), seqs
        int32 [B] (default: sequence b).  scale defaults to head_dim ** -0.5.
        Returns out, or (out, lse) with return_lse or lse.  workspace: a uint8
        tensor of at least workspace_bytes(B, n_heads) (default: allocated)."""
        if stream is not None:
            return self._call(stream, self.decode, q, lens, seqs, window, sinks, scale, out, lse, return_lse, workspace)
        return self._t.decode(self._cache, q, lens, seqs, window, sinks, scale, out, lse, return_lse, workspace)

    def decode_shared(self, q, lens, groups, shared, prefixes, seqs=None, scale=None, out=None, lse=None,
                      return_lse=False, workspace=None, stream=None):
        """decode() for groups of sequences that share a long prefix, read once for all of a group: rows groups[i] ..
        groups[i + 1] - 1 of q find their first shared[i] keys in the pages of table row prefixes[i] and the others in
        their own (seqs[b], default b).  groups int32 [n_groups + 1], shared and prefixes int32 [n_groups]; lens counts
        all keys of a row.  workspace: a uint8 tensor of at least shared_workspace_bytes(B, n_heads, n_groups)."""
        if stream is not None:
            return self._call(stream, self.decode_shared, q, lens, groups, shared, prefixes, seqs, scale, out, lse,
                              return_lse, workspace)
        return self._t.decode_shared(self._cache, q, lens, groups, shared, prefixes, seqs, scale, out, lse, return_lse,
                                     workspace)

    def prefill(self, q, cu, lens, seqs=None, window=0, sinks=0, scale=None, out=None, lse=None, return_lse=False,
                stream=None):
        """Attention of several tokens per sequence: rows cu[b] .. cu[b + 1] - 1
        of q [n, n_heads, head_dim] are the last positions of sequence b (or
        seqs[b]), which holds lens[b] keys.  cu int32 [B + 1], lens int32 [B]."""
        if stream is not None:
            return self._call(stream, self.prefill, q, cu, lens, seqs, window, sinks, scale, out, lse, return_lse)
        return self._t.prefill(self._cache, q, cu, lens, seqs, window, sinks, scale, out, lse, return_lse)

    def workspace_bytes(self, B: int, n_heads: int) -> int:
        """Bytes of decode's workspace for B sequences of n_heads query heads (0: none is needed)."""
        return self._t.workspace_bytes(self._cache, B, n_heads)

    def shared_workspace_bytes(self, B: int, n_heads: int, n_groups: int) -> int:
        """The same of decode_shared's."""
        return self._t.shared_workspace_bytes(self._cache, B, n_heads, n_groups)

    def sync_status(self, stream=None) -> int:
        """Wait for the stream, return and clear the first device-side error (0: none).  What calls on
        other streams raise meanwhile is returned now or by the next sync_status, never lost."""
        stream = torch.cuda.current_stream(self.device) if stream is None else stream
        with self._on(stream):
            return _take_status(self.status, stream)


def _status_word(device):
    """An int32 on the device, zero before any stream uses it."""
    with torch.cuda.device(device):
        status = torch.zeros(1, dtype=torch.int32, device=device)
        torch.cuda.current_stream().synchronize()
    return status


def _take_status(status, stream) -> int:
    taken = torch.empty(1, dtype=torch.int32, device=stream.device)
    E.check(E.ember_paged_take_status(_ptr(status), _ptr(taken), _stream_ptr(stream)), "ember_paged_take_status")
    return int(taken.item())


class Adapters:
    """Low-rank adapters of one projection, for batches whose rows name different ones (include/ember.h,
    "projections with adapters").

    a      bf16 or f16 [n_adapters, rank, K]; rank a multiple of 8 up to 128
    b      the same type, [n_adapters, N, rank]
    scale  f32 [n_adapters] (default: 1 each)

    All contiguous and the caller's; they may change between calls, and be moved to other storage of the same type,
    shape and device (t.data = ..), but not be replaced: the attributes are read-only.  Streams, gradients and errors as in PagedKV:
    calls are asynchronous on `stream` (default: the current one), tensors that require a gradient are refused
    unless gradients are off, device-side errors are read with sync_status().
    """

    def __init__(self, a, b, scale=None):
        for t, what in ((a, "a"), (b, "b")):
            if not isinstance(t, torch.Tensor) or not t.is_cuda:
                raise ValueError(f"{what} must be a tensor on a CUDA device")
        self._abs, self.device = (a, b, scale), a.device
        self.status = _status_word(self.device)
        self._t = _rows_torch()
        with torch.cuda.device(self.device):
            self._adapters = self._t.adapters(a, b, scale, self.status)

    a, b, scale = (property(lambda self, i=i: self._abs[i]) for i in range(3))

    def project(self, x, w, ids, bias=None, out=None, out_dtype=None, workspace=None, stream=None):
        """x [n, K] through the projection w [N, K] (+ bias [N]) with the adapter ids[i] of row i beside it (int32
        [n]; negative: none).  x, w and bias have the adapters' type.  Returns out [n, N] of that type, or of
        out_dtype = torch.float32.  workspace: a uint8 tensor of at least workspace_bytes(n) (default: allocated)."""
        if stream is None:
            return self._t.project(self._adapters, x, w, ids, bias, out, out_dtype, workspace)
        if stream.device != self.device:
            raise ValueError(f"the stream belongs to {stream.device}, the adapters to {self.device}")
        with torch.cuda.stream(stream):
            r = self._t.project(self._adapters, x, w, ids, bias, out, out_dtype, workspace)
        _keep_for(stream, x, w, ids, bias, out, workspace, self.a, self.b, self.scale)
        return r

    def workspace_bytes(self, n: int) -> int:
        """Bytes of project's workspace for n rows."""
        return E.ember_adapter_workspace(n, self.a.shape[1])

    def sync_status(self, stream=None) -> int:
        """Wait for the stream, return and clear the first device-side error (0: none), as in PagedKV."""
        stream = torch.cuda.current_stream(self.device) if stream is None else stream
        if stream.device != self.device:
            raise ValueError(f"the stream belongs to {stream.device}, the adapters to {self.device}")
        with torch.cuda.stream(stream):
            return _take_status(self.status, stream)


class Logprobs(typing.NamedTuple):
    """What logprobs() returns, a row of logits each."""

    logprob: torch.Tensor | None       # f32 [n]: of the given token (None without ids)
    rank: torch.Tensor | None          # int32 [n]: tokens that stand before it
    entropy: torch.Tensor              # f32 [n]
    top_ids: torch.Tensor              # int32 [n, top]: the most probable tokens, the first first
    top_logprobs: torch.Tensor         # f32 [n, top]


def logprobs(logits, ids=None, top: int = 0, temperature: float = 1.0, stream=None) -> Logprobs:
    """Log probabilities of given tokens with their ranks, the entropy, and the `top` (at most 32) most probable
    tokens (include/ember.h, "log probabilities").

    logits f32, bf16 or f16 [n, V], rows of any stride; ids int32 [n].  Tokens stand in the order of their logits,
    equal ones in that of their indices.  Asynchronous on `stream` (default: the current stream of the logits'
    device) under the rules of PagedKV.  It has no gradient: logits that require one are refused unless gradients
    are off."""
    if stream is not None:
        if stream.device != logits.device:
            raise ValueError(f"the stream belongs to {stream.device}, the logits to {logits.device}")
        with torch.cuda.stream(stream):
            r = logprobs(logits, ids, top, temperature)
        _keep_for(stream, logits, ids)
        return r
    return Logprobs(*_rows_torch().logprobs(logits, ids, top, temperature))


def _keep_for(stream, *args):
    """What a call on another stream reads and writes stays allocated until it has run there."""
    for t in args:
        if isinstance(t, torch.Tensor):
            t.record_stream(stream)


_PAGE_DTYPES = {torch.bfloat16: E.BF16, torch.float16: E.F16}
_torch_sides = {}


def _torch_side(name, build, entries):
    """A compiled marshalling module (csrc/<name>.cpp), on the loaded library's entry points."""
    if name not in _torch_sides:
        lib = E.load()
        spec = importlib.util.spec_from_file_location(name, build())
        t = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(t)
        t.entries(*(C.cast(getattr(lib, n), C.c_void_p).value for n in (*entries, "ember_last_error")), E.EmberError)
        _torch_sides[name] = t
    return _torch_sides[name]


def _paged_torch():
    return _torch_side("paged_torch", E._build.build_ext,
                       ("ember_paged_append", "ember_paged_decode", "ember_paged_decode_workspace", "ember_paged_prefill",
                        "ember_paged_decode_shared", "ember_paged_decode_shared_workspace"))


def _rows_torch():
    return _torch_side("rows_torch", E._build.build_rows_ext,
                       ("ember_logprobs", "ember_adapter_project", "ember_adapter_workspace"))


def _wrap_device(ptr: int, nbytes: int, device) -> torch.Tensor:
    """A uint8 tensor viewing nbytes of device memory owned by the library."""
    class _Holder:
        pass

    h = _Holder()
    h.__cuda_array_interface__ = {"shape": (nbytes,), "typestr": "|u1", "data": (ptr, False),
                                  "version": 3, "strides": None}
    return torch.as_tensor(h, device=device)
