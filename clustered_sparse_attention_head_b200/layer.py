"""Python front end of the calls around the attention (ac_layer_*), with the
same call names as the C ABI.

``AttnLayer`` owns one ``ac_layer`` and a workspace.  It checks tensors' types,
devices and shapes, takes views of any token and head strides (a slice of the
packed projection needs no copy) and allocates outputs with torch; the work is
the library's kernels.
"""
from __future__ import annotations

import ctypes
import struct
from ctypes import byref, c_void_p
from dataclasses import dataclass

import torch

from . import _abi
from ._abi import check

_NORMS = {"none": _abi.AC_NORM_NONE, "rms": _abi.AC_NORM_RMS, "layer": _abi.AC_NORM_LAYER}
_LAYOUTS = {"interleaved": _abi.AC_ROPE_INTERLEAVED, "half": _abi.AC_ROPE_HALF}
_SCALINGS = {"none": _abi.AC_ROPE_PLAIN, "linear": _abi.AC_ROPE_LINEAR, "ntk": _abi.AC_ROPE_NTK,
             "yarn": _abi.AC_ROPE_YARN}
_DTYPES = {"bf16": (_abi.AC_BF16, torch.bfloat16), "f32": (_abi.AC_F32, torch.float32)}
_view = struct.Struct("Qqqq").pack  # an ac_tensor as bytes, which ctypes passes by address


def _int32(v):
    """A bound as a C int, which ctypes would take modulo 2^32."""
    return min(max(int(v), -1 << 31), (1 << 31) - 1)


@dataclass
class LayerConfig:
    heads: int
    d: int
    kv_heads: int | None = None      # None: heads
    dtype: str = "bf16"              # "bf16" | "f32"
    w_dtype: str | None = None       # norm weights; None: dtype
    norm: str = "rms"                # "none" | "rms" | "layer"
    eps: float = 1e-6
    rope_dims: tuple = ()            # rotated elements per axis; () = no rotation
    rope_max: tuple = ()             # positions per axis (the latent grid)
    rope_layout: str = "interleaved"  # | "half"
    rope_theta: float = 10000.0
    rope_scaling: str = "none"       # | "linear" | "ntk" | "yarn"
    rope_factor: float = 1.0
    rope_orig: int = 0
    rope_beta_fast: float = 32.0
    rope_beta_slow: float = 1.0
    page_size: int = 0               # tokens per cache page; 0 = no cache
    causal_block: int = 0            # 0: all keys; 1: causal by token; B: causal by blocks of B tokens
    window: int = 0                  # > 0: only the last `window` positions
    scale: float = 0.0               # 0: 1 / sqrt(d)

    def __post_init__(self):
        self.kv_heads = self.heads if self.kv_heads is None else self.kv_heads
        self.w_dtype = self.w_dtype or self.dtype

    def to_c(self) -> _abi.ac_layer_config:
        def pick(table, key, what):
            if key not in table:
                raise ValueError(f"LayerConfig: {what} must be one of {sorted(table)}, not {key!r}")
            return table[key]

        if len(self.rope_dims) != len(self.rope_max) or len(self.rope_dims) > 3:
            raise ValueError("LayerConfig: rope_dims and rope_max take one number per axis, at most three")
        for name in ("heads", "kv_heads", "d", "rope_dims", "rope_max", "rope_orig", "page_size", "causal_block", "window"):
            v = getattr(self, name)
            if any(_int32(x) != x for x in (v if name in ("rope_dims", "rope_max") else (v,))):
                raise ValueError(f"LayerConfig: {name} must be 32-bit integers, not {v!r}")
        dims = (ctypes.c_int * 3)(*self.rope_dims)
        top = (ctypes.c_int * 3)(*self.rope_max)
        return _abi.ac_layer_config(
            self.heads, self.kv_heads, self.d,
            pick(_DTYPES, self.dtype, "dtype")[0], pick(_DTYPES, self.w_dtype, "w_dtype")[0],
            pick(_NORMS, self.norm, "norm"), float(self.eps), len(self.rope_dims), dims, top,
            pick(_LAYOUTS, self.rope_layout, "rope_layout"), float(self.rope_theta),
            pick(_SCALINGS, self.rope_scaling, "rope_scaling"), float(self.rope_factor), int(self.rope_orig),
            float(self.rope_beta_fast), float(self.rope_beta_slow), self.page_size, self.causal_block, self.window,
            float(self.scale))


class _NormRope(torch.autograd.Function):
    """ac_qk_norm_rope in torch's graph: ac_qk_norm_rope_backward on the way back."""

    @staticmethod
    def forward(ctx, layer, table, pos, stream, q, k, w_q, w_k, b_q, b_k):
        ctx.layer = layer
        ctx.set_materialize_grads(False)
        x = (q, k, w_q, w_k, b_q, b_k) if layer.normed else (None,) * 6  # a rotation's gradient needs none of them
        ctx.save_for_backward(table, pos, *x)
        return layer.ac_qk_norm_rope(q, k, table, pos, w_q, w_k, b_q, b_k, stream=stream)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gq, gk):
        table, pos, q, k, w_q, w_k, b_q, b_k = ctx.saved_tensors
        need = ctx.needs_input_grad[4:]
        gq = gq if need[0] or need[2] or need[4] else None
        gk = gk if need[1] or need[3] or need[5] else None
        if gq is None and gk is None:
            return (None,) * 10
        r = ctx.layer.ac_qk_norm_rope_backward(_readable(gq), _readable(gk), q, k, table, pos, w_q, w_k, b_q, b_k)
        return (None,) * 4 + tuple(r[n] for n in ("q", "k", "w_q", "w_k", "b_q", "b_k"))


def _readable(g):
    """A gradient whose strides and alignment the calls take: torch hands on
    any, a sum's with strides of 0 among them."""
    if g is None or (g.stride(-1) == 1 and g.data_ptr() % 16 == 0 and
                     all(s * g.element_size() % 16 == 0 and s < 1 << 31 for s in g.stride()[:-1])):
        return g
    return g.clone(memory_format=torch.contiguous_format)


class AttnLayer:
    """One attention layer's calls.  ``device``: the GPU of every tensor passed
    in.  Calls that use the workspace (ac_qk_norm_rope_backward, ac_cache_attn)
    must not overlap on the GPU with another such call of the same layer.

    ``stream=`` runs a call on another stream than the current one.  Its
    inputs must be ready there, and what it returns must be waited for before
    it is used elsewhere (``wait_stream`` both ways); it may be freed at any time.

    A CUDA graph that captured calls writes to the layer's status block and
    workspace: keep the layer for as long as the graph."""

    def __init__(self, cfg: LayerConfig, device="cuda", workspace: torch.Tensor | None = None):
        self.cfg = cfg
        self._layer = c_void_p()
        self.lib = _abi.load()
        device = torch.device(device)
        self.device = torch.device("cuda", torch.cuda.current_device()) if device.index is None else device
        c = cfg.to_c()
        with torch.cuda.device(self.device):
            check("ac_layer_create", self.lib.ac_layer_create(byref(c), byref(self._layer)))
        self.heads, self.kv_heads, self.d, self.axes = c.heads, c.kv_heads, c.d, c.rope_axes
        self._w_shape = (c.d,)
        self.normed = c.norm != _abi.AC_NORM_NONE
        self.dtype, self.w_dtype = _DTYPES[cfg.dtype][1], _DTYPES[cfg.w_dtype][1]
        self._index = self.device.index
        # allocations of these types begin from an empty tensor
        self._f32 = torch.empty(0, dtype=torch.float32, device=self.device)
        self._like_w = self._f32.to(self.w_dtype)
        nb = ctypes.c_size_t()
        self._pairs = 0
        if self.axes:
            check("ac_rope_table_size", self.lib.ac_rope_table_size(self._layer, byref(nb)))
            self._pairs = nb.value // 8
        check("ac_layer_workspace_size", self.lib.ac_layer_workspace_size(self._layer, byref(nb)))
        self.ws_bytes = nb.value
        if workspace is None:
            workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
            # the block may still be in use on the current stream; calls may come on any
            torch.cuda.current_stream(self.device).synchronize()
        elif workspace.device != self.device or not workspace.is_contiguous():
            raise ValueError("AttnLayer: workspace must be a contiguous tensor on the layer's device")
        self.ws = workspace
        self._ws_have = workspace.numel() * workspace.element_size()
        self._ws_ptr = workspace.data_ptr()

    def close(self):
        if self._layer:
            self.lib.ac_layer_destroy(self._layer)
            self._layer = c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # --------------------------------------------------------------- helpers
    # The calls are a few microseconds on the GPU for few tokens, so these keep
    # to the cheapest forms that check everything.
    def _rows(self, t, name, tokens, heads):
        """The ac_tensor of a [tokens, heads, d] view."""
        if t.dtype != self.dtype or t.get_device() != self._index or t.shape != (tokens, heads, self.d):
            self._refuse(t, name, (tokens, heads, self.d))
        sn, sh, one = t.stride()
        if one != 1:
            raise ValueError(f"{name}: the last dimension must be contiguous")
        return _view(t.data_ptr(), 0, sn, sh)

    def _bnhd(self, t, name, batch, n, heads):
        """... of a [batch, n, heads, d] view."""
        if t.dtype != self.dtype or t.get_device() != self._index or t.shape != (batch, n, heads, self.d):
            self._refuse(t, name, (batch, n, heads, self.d))
        sb, sn, sh, one = t.stride()
        if one != 1:
            raise ValueError(f"{name}: the last dimension must be contiguous")
        return _view(t.data_ptr(), sb, sn, sh)

    def _bhnd(self, t, name, batch, n, heads):
        """... of a [batch, heads, n, d] view."""
        if t.dtype != self.dtype or t.get_device() != self._index or t.shape != (batch, heads, n, self.d):
            self._refuse(t, name, (batch, heads, n, self.d))
        sb, sh, sn, one = t.stride()
        if one != 1:
            raise ValueError(f"{name}: the last dimension must be contiguous")
        return _view(t.data_ptr(), sb, sn, sh)

    def _refuse(self, t, name, shape):
        raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)} on {t.device}, expected {self.dtype} {shape} on "
                         f"{self.device}")

    def _plain(self, t, name, dtype, shape):
        """Pointer of a contiguous tensor."""
        if t.dtype != dtype or t.get_device() != self._index or t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)} on {t.device}, expected contiguous {dtype} {shape} "
                             f"on {self.device}")
        return t.data_ptr()

    def _w(self, t, name):
        if t is None:
            return None
        if t.dtype != self.w_dtype or t.get_device() != self._index or t.shape != self._w_shape or t.stride() != (1,):
            return self._plain(t, name, self.w_dtype, self._w_shape)
        return t.data_ptr()

    def _table(self, t):
        if t is None:
            if self.axes:
                raise ValueError("table: this layer rotates, pass the tensor of ac_rope_table()")
            return None
        return self._plain(t, "table", torch.float32, (self._pairs, 2))

    def _pos(self, t, batch, n):
        """Pointer and batch stride of [n, axes] or [batch, n, axes] positions."""
        if t is None:
            return None, 0
        if t.dim() == 3:
            return self._plain(t, "pos", torch.int32, (batch, n, self.axes)), n * self.axes
        return self._plain(t, "pos", torch.int32, (n, self.axes)), 0

    def _new(self, like, shape, stream):
        """An uninitialised output of `like`'s type for a call on `stream`.  It is
        allocated on that stream: a block freed on the current one may still
        be in use there.  The current stream is recorded, so that freeing the
        output does not hand its memory out while the caller reads it."""
        if stream is None:
            return like.new_empty(shape)
        with torch.cuda.stream(stream):
            t = like.new_empty(shape)
        t.record_stream(torch.cuda.current_stream(self.device))
        return t

    def _call(self, fn, stream, tensors, *args):
        """The C call on `stream` (default: the current stream of the layer's
        device).  Tensors used on another stream than the current one are
        recorded there, so that freeing them does not hand their memory out
        while the call runs."""
        if torch._C._cuda_getDevice() != self._index:
            with torch.cuda.device(self.device):
                return self._call(fn, stream, tensors, *args)
        raw = torch._C._cuda_getCurrentRawStream(self._index)
        if stream is not None and stream.cuda_stream != raw:
            raw = stream.cuda_stream
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
        code = getattr(self.lib, fn)(self._layer, *args, raw)
        if code:
            check(fn, code)

    def get_status(self, stream=None) -> int:
        with torch.cuda.device(self.device):
            s = stream if stream is not None else torch.cuda.current_stream()
            return self.lib.ac_layer_get_status(self._layer, s.cuda_stream)

    # ------------------------------------------------------------- the calls
    def ac_rope_table(self, stream=None):
        """The layer's cosines and sines, [pairs of all axes, 2] fp32: made once,
        passed to the calls below."""
        if not self.axes:
            check("ac_rope_table", _abi.AC_ERR_UNSUPPORTED)
        table = self._new(self._f32, (self._pairs, 2), stream)
        self._call("ac_rope_table", stream, (table,), table.data_ptr())
        return table

    def ac_qk_norm_rope(self, q, k, table=None, pos=None, w_q=None, w_k=None, b_q=None, b_k=None, q_out=None,
                        k_out=None, stream=None):
        """Norm and rotation of q [batch, n, heads, d] and k [batch, n, kv_heads, d]
        (views of any strides; either may be None).  Returns (q_out, k_out) in
        the attention's layout [batch, heads, n, d] unless given; given outputs
        are [batch, heads, n, d] views too, and q_out = q.transpose(1, 2) works
        in place.  Under autograd the outputs carry the gradients of
        ac_qk_norm_rope_backward to inputs, weights and biases that ask for them
        (given outputs cannot; the cache's calls have no gradients)."""
        if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (q, k, w_q, w_k, b_q, b_k)):
            if q_out is not None or k_out is not None:
                raise ValueError("ac_qk_norm_rope: q_out and k_out do not join torch's graph, but an input requires a "
                                 "gradient; call it under torch.no_grad()")
            return _NormRope.apply(self, table, pos, stream, q, k, w_q, w_k, b_q, b_k)
        ref = q if q is not None else k
        if ref is None or ref.dim() != 4:
            raise ValueError("ac_qk_norm_rope: q or k [batch, n, heads, d] is required")
        batch, n, _, d = ref.shape
        xq = yq = xk = yk = None
        if q is not None:
            if q_out is None:
                q_out = self._new(q, (batch, self.heads, n, d), stream)
            xq, yq = self._bnhd(q, "q", batch, n, self.heads), self._bhnd(q_out, "q_out", batch, n, self.heads)
        elif q_out is not None:
            raise ValueError("q_out without q")
        if k is not None:
            if k_out is None:
                k_out = self._new(k, (batch, self.kv_heads, n, d), stream)
            xk, yk = self._bnhd(k, "k", batch, n, self.kv_heads), self._bhnd(k_out, "k_out", batch, n, self.kv_heads)
        elif k_out is not None:
            raise ValueError("k_out without k")
        pos_p, pos_stride = self._pos(pos, batch, n)
        self._call("ac_qk_norm_rope", stream, (q, k, table, pos, w_q, w_k, b_q, b_k, q_out, k_out), batch, n,
                   self._table(table), pos_p, pos_stride, xq, self._w(w_q, "w_q"), self._w(b_q, "b_q"), yq, xk,
                   self._w(w_k, "w_k"), self._w(b_k, "b_k"), yk)
        return q_out, k_out

    def ac_qk_norm_rope_backward(self, gq, gk, q=None, k=None, table=None, pos=None, w_q=None, w_k=None, b_q=None,
                                 b_k=None, dq=None, dk=None, stream=None):
        """Gradients of ac_qk_norm_rope: gq [batch, heads, n, d], gk [batch,
        kv_heads, n, d] and the forward call's inputs.  Returns a dict: "q", "k"
        [batch, n, heads, d] (dq, dk if given), "w_q", "b_q", "w_k", "b_k" (None
        where the forward call had no such weight)."""
        ref = gq if gq is not None else gk
        if ref is None or ref.dim() != 4:
            raise ValueError("ac_qk_norm_rope_backward: gq or gk [batch, heads, n, d] is required")
        batch, n = ref.shape[0], ref.shape[2]
        pos_p, pos_stride = self._pos(pos, batch, n)
        sums = self._new(self._like_w, (4, self.d), stream).unbind() if self.normed else ()
        aq, rq = self._back_args(gq, q, w_q, b_q, dq, sums[:2], batch, n, self.heads, "q", stream)
        ak, rk = self._back_args(gk, k, w_k, b_k, dk, sums[2:], batch, n, self.kv_heads, "k", stream)
        self._call("ac_qk_norm_rope_backward", stream, (gq, q, w_q, *rq, gk, k, w_k, *rk, table, pos, self.ws), batch,
                   n, self._table(table), pos_p, pos_stride, *aq, *ak, self._ws_ptr, self._ws_have)
        return {"q": rq[0], "w_q": rq[1], "b_q": rq[2], "k": rk[0], "w_k": rk[1], "b_k": rk[2]}

    def _back_args(self, g, x, w, b, dx, sums, batch, n, heads, name, stream):
        """One tensor's arguments of the backward call, and its (dx, dw, db);
        sums: where dw and db go."""
        if g is None:
            if dx is not None:
                raise ValueError(f"d{name} without g{name}")
            return (None,) * 6, (None, None, None)
        xv = dw = db = None
        if self.normed:
            if x is None:
                raise ValueError(f"{name}: the norm's gradient needs the forward call's input")
            xv = self._bnhd(x, name, batch, n, heads)
            if w is not None:
                dw = sums[0]
            if b is not None:
                self._w(b, "b_" + name)
                db = sums[1]
        if dx is None:
            dx = self._new(g, (batch, n, heads, self.d), stream)
        return ((self._bhnd(g, "g" + name, batch, n, heads), xv, self._w(w, "w_" + name),
                 self._bnhd(dx, "d" + name, batch, n, heads), None if dw is None else dw.data_ptr(),
                 None if db is None else db.data_ptr()), (dx, dw, db))

    def _cache(self, tokens, k_pages, v_pages, block_table, q_start, kv_len):
        """The arguments that both cache calls share."""
        seqs = kv_len.shape[0]
        num_pages = k_pages.shape[0]
        pool = (num_pages, self.kv_heads, self.cfg.page_size, self.d)
        if block_table.dim() != 2:
            raise ValueError("block_table: [sequences, pages] is required")
        max_pages = block_table.shape[1]
        return (seqs, tokens, self._plain(q_start, "q_start", torch.int32, (seqs + 1,)),
                self._plain(kv_len, "kv_len", torch.int32, (seqs,)),
                self._plain(block_table, "block_table", torch.int32, (seqs, max_pages)), max_pages, num_pages,
                self._plain(k_pages, "k_pages", self.dtype, pool), self._plain(v_pages, "v_pages", self.dtype, pool))

    def ac_cache_append(self, k, v, k_pages, v_pages, block_table, q_start, kv_len, q=None, table=None, pos=None,
                        w_q=None, w_k=None, b_q=None, b_k=None, q_out=None, stream=None):
        """Writes the new tokens' keys (normed, rotated) and values [tokens,
        kv_heads, d] to their pages; with q [tokens, heads, d] returns the normed
        and rotated queries (q_out if given), else None.  On one axis without
        pos, tokens past the table stay unrotated and set the status word."""
        tokens = k.shape[0]
        seqs, _, qs, kl, bt, max_pages, num_pages, kp, vp = self._cache(tokens, k_pages, v_pages, block_table,
                                                                        q_start, kv_len)
        pos_p = None if pos is None else self._plain(pos, "pos", torch.int32, (tokens, self.axes))
        qv = qo = None
        if q is not None:
            qv = self._rows(q, "q", tokens, self.heads)
            if q_out is None:
                q_out = self._new(q, (tokens, self.heads, self.d), stream)
            qo = self._rows(q_out, "q_out", tokens, self.heads)
        elif q_out is not None:
            raise ValueError("q_out without q")
        self._call("ac_cache_append", stream,
                   (k, v, k_pages, v_pages, block_table, q_start, kv_len, q, table, pos, w_q, w_k, b_q, b_k, q_out),
                   seqs, tokens, qs, kl, bt, max_pages, num_pages, self._table(table), pos_p,
                   self._rows(k, "k", tokens, self.kv_heads), self._w(w_k, "w_k"), self._w(b_k, "b_k"),
                   self._rows(v, "v", tokens, self.kv_heads), kp, vp, qv, self._w(w_q, "w_q"), self._w(b_q, "b_q"), qo)
        return q_out

    def ac_cache_attn(self, q, k_pages, v_pages, block_table, q_start, kv_len, max_q=None, max_kv=None, out=None,
                      lse=False, stream=None):
        """Attention of the new tokens q [tokens, heads, d] over the cache.
        max_q, max_kv: bounds on any sequence's new tokens and length (default:
        what the tensors' shapes allow); tight bounds let short batches use the
        whole GPU.  Returns out [tokens, heads, d], with lse=True (out, lse
        [tokens, heads] fp32)."""
        tokens = q.shape[0]
        seqs, _, qs, kl, bt, max_pages, num_pages, kp, vp = self._cache(tokens, k_pages, v_pages, block_table,
                                                                        q_start, kv_len)
        if out is None:
            out = self._new(q, (tokens, self.heads, self.d), stream)
        lse_t = self._new(self._f32, (tokens, self.heads), stream) if lse else None
        self._call("ac_cache_attn", stream, (q, k_pages, v_pages, block_table, q_start, kv_len, out, lse_t, self.ws),
                   seqs, tokens, tokens if max_q is None else _int32(max_q),
                   _int32(max_pages * self.cfg.page_size if max_kv is None else max_kv), qs, kl, bt, max_pages, num_pages,
                   self._rows(q, "q", tokens, self.heads), kp, vp, self._rows(out, "out", tokens, self.heads),
                   None if lse_t is None else lse_t.data_ptr(),
                   self._ws_ptr, self._ws_have)
        return (out, lse_t) if lse else out
