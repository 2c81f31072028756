"""Runners for what stands between the recurrent layers of a hybrid model: attention over
a paged key-value cache, and the residual add with its RMS norm.

As the runners in decoder.py, each owns the device buffers of one layer (or uses tensors
that the caller hands in), a step is a sequence of librssm calls in stream order, and no
call synchronises, so a step can be captured in a CUDA graph:

  attention:  rssm_attn_append -> rssm_attn_decode -> rssm_attn_advance
              (T > 1 drafts: append and decode, then advance by the accepted counts)
  norm:       rssm_add_rmsnorm
"""
import ctypes

import torch

from . import _binding as B
from .decoder import torch_dtype_code

__all__ = ["PagedAttentionDecoder", "AddRMSNorm"]


def _code(dt):
    return B.RSSM_E4M3 if dt == torch.float8_e4m3fn else torch_dtype_code(dt)


def _check(name, t, shape, dtype, device):
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != device or \
            not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor %s on %s" % (name, dtype, tuple(shape),
                                                                         device))
    return t


def _device(device):
    """The device meant: the current GPU for None and for "cuda" without a number."""
    dev = torch.device("cuda" if device is None else device)
    if dev.type == "cuda" and dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    return dev


def _index(device):
    """What get_device() says of a tensor on this device."""
    return device.index if device.type == "cuda" else -1


def _check_out(name, t, count, dtype, index):
    if t.dtype is not dtype or t.numel() != count or not t.is_contiguous() or \
            t.get_device() != index:
        raise ValueError("%s must be dense, %d %s values on the runner's device"
                         % (name, count, dtype))
    return t.data_ptr()


def _check_list(name, t, count, index):
    if t is None:
        return None
    if t.dtype is not torch.int32 or t.shape[0] != count or not t.is_contiguous() or \
            t.get_device() != index:
        raise ValueError("%s must be a dense int32 list of %d on the runner's device"
                         % (name, count))
    return t.data_ptr()


class _Fixed:
    """Calls pass addresses that were taken once, so a runner's tensors and sizes stay the
    ones it was made with: new values are copied into them."""
    _free = ()

    def __setattr__(self, name, value):
        if "_plans" in self.__dict__ and name not in self._free and name[0] != "_":
            raise AttributeError("%s is fixed when the runner is made; copy into its tensors" % name)
        object.__setattr__(self, name, value)


class PagedAttentionDecoder(_Fixed):
    """Attention decode for one layer over a paged cache.

    Buffers: k_cache, v_cache [num_pages, HKV, page_size, D] (cache_dtype: bfloat16 or
    float8_e4m3fn), k_scale, v_scale [num_pages, HKV, page_size] float32 (8-bit cache
    only), page_table [num_slots, max_pages] int32 (-1: no page yet; the caller assigns
    pages), slot_len [num_slots] int32, and workspace / o / lse for up to max_batch rows of
    T query tokens. Any of the caches, the scales, page_table and slot_len can be the
    caller's tensors (page_table and slot_len are commonly shared by a model's layers). scale
    and window may be set between calls."""

    _free = ("scale", "window")

    def __init__(self, num_q_heads, num_kv_heads, head_dim, page_size, num_pages, num_slots,
                 max_pages, max_batch, T=1, act_dtype=torch.bfloat16, cache_dtype=torch.bfloat16,
                 out_dtype=torch.bfloat16, window=0, scale=None, device=None, k_cache=None,
                 v_cache=None, k_scale=None, v_scale=None, page_table=None, slot_len=None):
        dev = _device(device)
        self.HQ, self.HKV, self.D, self.T = num_q_heads, num_kv_heads, head_dim, T
        self.page_size, self.num_pages, self.max_pages = page_size, num_pages, max_pages
        self.num_slots, self.max_batch, self.window = num_slots, max_batch, window
        self.scale = head_dim ** -0.5 if scale is None else scale
        self.act_dtype, self.cache_dtype, self.out_dtype = act_dtype, cache_dtype, out_dtype
        self.device = dev

        def buf(name, given, shape, dtype, fill=0):
            if given is None:
                # 8-bit caches are filled through their bytes
                raw = torch.uint8 if dtype == torch.float8_e4m3fn else dtype
                return torch.full(shape, fill, device=dev, dtype=raw).view(dtype)
            return _check(name, given, shape, dtype, dev)
        pages = (num_pages, num_kv_heads, page_size)
        self.k_cache = buf("k_cache", k_cache, pages + (head_dim,), cache_dtype)
        self.v_cache = buf("v_cache", v_cache, pages + (head_dim,), cache_dtype)
        if cache_dtype == torch.float8_e4m3fn:
            self.k_scale = buf("k_scale", k_scale, pages, torch.float32)
            self.v_scale = buf("v_scale", v_scale, pages, torch.float32)
        else:
            self.k_scale = self.v_scale = None
        self.page_table = buf("page_table", page_table, (num_slots, max_pages), torch.int32, -1)
        self.slot_len = buf("slot_len", slot_len, (num_slots,), torch.int32)
        self.dev_err = torch.zeros(4, device=dev, dtype=torch.int32)
        self.cache = B.attn_cache(self.k_cache, self.v_cache, self.k_scale, self.v_scale,
                                  self.page_table, self.slot_len)
        self.ws_bytes = B.rssm_attn_workspace_size(self.dims(max_batch))
        # zero-filled: the decode call keeps its arrival counters here
        self.workspace = torch.zeros(max(self.ws_bytes, 16), device=dev, dtype=torch.uint8)
        self.o = torch.empty(max_batch, T, num_q_heads, head_dim, device=dev, dtype=out_dtype)
        self.lse = torch.empty(max_batch, T, num_q_heads, device=dev, dtype=torch.float32)
        # what every call passes, made once
        self._append, self._read = B.entry("rssm_attn_append"), B.entry("rssm_attn_read")
        self._decode, self._advance = B.entry("rssm_attn_decode"), B.entry("rssm_attn_advance")
        self._cache = ctypes.byref(self.cache)
        self._ws, self._err = self.workspace.data_ptr(), self.dev_err.data_ptr()
        self._index = _index(self.workspace.device)
        self._plans = {}

    def dims(self, batch):
        return B.AttnDims(batch, self.T, self.HQ, self.HKV, self.D, self.page_size, self.num_pages,
                          self.max_pages, self.num_slots, torch_dtype_code(self.act_dtype),
                          _code(self.cache_dtype), torch_dtype_code(self.out_dtype))

    def _plan(self, cache_indices):
        """What calls of b rows share: a reference to their dims, q's element count, the
        outputs and their addresses. Kept, because a small call's time is the host's."""
        b = cache_indices.shape[0]
        if cache_indices.dtype is not torch.int32 or not cache_indices.is_contiguous() or \
                cache_indices.get_device() != self._index:
            raise ValueError("cache_indices must be a dense int32 list on the runner's device")
        p = self._plans.get(b)
        if p is None:
            o, lse = self.o[:b], self.lse[:b]
            p = self._plans[b] = (ctypes.byref(self.dims(b)), b * self.T * self.HQ * self.D, o, lse,
                                  o.data_ptr(), lse.data_ptr())
        return p

    def _stride(self, name, t, heads):
        """Element distance between consecutive tokens of t [tokens, heads, D] or
        [rows, T, heads, D]."""
        if t.get_device() != self._index:
            raise ValueError("%s is not on the runner's device" % name)
        if t.dtype is self.act_dtype and t.is_contiguous() and t.shape[-2] == heads and \
                t.shape[-1] == self.D:
            return heads * self.D
        s, n = t.stride(), t.shape
        if t.dtype != self.act_dtype or n[-2:] != (heads, self.D) or s[-1] != 1 or \
                (s[-2] != self.D and heads > 1) or \
                (len(n) == 4 and n[0] > 1 and n[1] > 1 and s[0] != n[1] * s[1]) or len(n) > 4:
            raise ValueError("%s: tokens of dense [%d, %d] %s blocks, evenly spaced, are wanted"
                             % (name, heads, self.D, self.act_dtype))
        return s[0] if len(n) == 3 or n[1] == 1 else s[1]

    def append(self, k, v, cache_indices, cu_tokens=None, stream=None):
        """Write new tokens' k, v [n, HKV, D] (or [b, T, HKV, D]) after the rows' committed
        tokens; cu_tokens [b + 1] int32 for rows of different token counts (else T each)."""
        n = k.numel() // (self.HKV * self.D)
        if v.shape != k.shape:
            raise ValueError("k and v must have one shape")
        rc = self._append(self._plan(cache_indices)[0], self._cache, n,
                          _check_list("cu_tokens", cu_tokens, cache_indices.shape[0] + 1,
                                      self._index),
                          k.data_ptr(), self._stride("k", k, self.HKV), v.data_ptr(),
                          self._stride("v", v, self.HKV), cache_indices.data_ptr(), self._err,
                          B._stream(stream))
        if rc:
            raise B.RSSMError("rssm_attn_append", rc)

    def decode(self, q, cache_indices, appended=True, o=None, lse=None, with_lse=False,
               stream=None):
        """Attention of q [b, T, HQ, D] over the rows' tokens. appended: the queries' own
        tokens are in the cache and visible (see rssm_attn_decode). Returns o [b, T, HQ, D],
        with with_lse also lse [b, T, HQ]."""
        dims, count, own_o, own_lse, o_ptr, lse_ptr = self._plan(cache_indices)
        if q.numel() != count or own_lse.shape[0] != cache_indices.shape[0]:
            raise ValueError("q must be [b, %d, %d, %d], b = len(cache_indices) <= %d"
                             % (self.T, self.HQ, self.D, self.max_batch))
        if o is None:
            o = own_o
        else:
            o_ptr = _check_out("o", o, count, self.out_dtype, self._index)
        if lse is not None:
            lse_ptr = _check_out("lse", lse, count // self.D, torch.float32, self._index)
        elif with_lse:
            lse = own_lse
        else:
            lse_ptr = None
        rc = self._decode(dims, self._cache, appended, self.scale, self.window, q.data_ptr(),
                          self._stride("q", q, self.HQ), cache_indices.data_ptr(), self._ws,
                          self.ws_bytes, o_ptr, lse_ptr, self._err, B._stream(stream))
        if rc:
            raise B.RSSMError("rssm_attn_decode", rc)
        return (o, lse) if with_lse else o

    def advance(self, cache_indices, num_accepted=None, cu_tokens=None, stream=None):
        """Commit the appended tokens (of T drafts: the first num_accepted[b])."""
        b = cache_indices.shape[0]
        rc = self._advance(self._plan(cache_indices)[0], self._cache,
                           _check_list("cu_tokens", cu_tokens, b + 1, self._index),
                           _check_list("num_accepted", num_accepted, b, self._index),
                           cache_indices.data_ptr(), self._err, B._stream(stream))
        if rc:
            raise B.RSSMError("rssm_attn_advance", rc)

    def step(self, q, k, v, cache_indices, o=None, stream=None):
        """One decode step for rows cache_indices (padding rows: -1): append, decode,
        advance. Returns o [b, T, HQ, D]."""
        self.append(k, v, cache_indices, stream=stream)
        o = self.decode(q, cache_indices, o=o, stream=stream)
        self.advance(cache_indices, stream=stream)
        return o

    def read(self, cache_indices, cu_tokens, n_tokens, first=None, k=None, v=None, stream=None):
        """Committed tokens back, dense: k, v [n_tokens, HKV, D] (out_dtype; new tensors unless
        given)."""
        shape = (n_tokens, self.HKV, self.D)
        for t in (k, v):
            if t is not None and (t.dtype is not self.out_dtype or t.shape != shape or
                                  not t.is_contiguous() or t.get_device() != self._index):
                raise ValueError("k and v: dense [%d, %d, %d] %s on the runner's device"
                                 % (shape + (self.out_dtype,)))
        if k is None:
            k = torch.empty(shape, device=self.device, dtype=self.out_dtype)
        if v is None:
            v = torch.empty(shape, device=self.device, dtype=self.out_dtype)
        b = cache_indices.shape[0]
        rc = self._read(self._plan(cache_indices)[0], self._cache, n_tokens,
                        _check_list("cu_tokens", cu_tokens, b + 1, self._index),
                        _check_list("first", first, b, self._index), cache_indices.data_ptr(),
                        k.data_ptr(), v.data_ptr(), self._err, B._stream(stream))
        if rc:
            raise B.RSSMError("rssm_attn_read", rc)
        return k, v

    def reset_slots(self, slots, stream=None):
        """Lengths back to 0 (the page table is the caller's)."""
        B.rssm_advance_cursors(B.RSSM_CURSOR_RESET, self.slot_len, None, None, slots, None, None,
                               slots.shape[0], self.num_slots, 1, 0, None, None, self.dev_err,
                               stream)


class AddRMSNorm(_Fixed):
    """Residual add and RMS norm for one place in a model: r = x + residual, y = r /
    sqrt(mean(r^2) + eps) * weight, for up to max_rows rows. With out_dtype float8_e4m3fn y
    comes with float32 scales [rows, cols / scale_group] ([rows, 1] for scale_group 0). eps may
    be set between calls."""

    _free = ("eps",)

    def __init__(self, weight, eps, max_rows, act_dtype=torch.bfloat16, out_dtype=torch.bfloat16,
                 scale_group=0, device=None):
        dev = _device(device)
        self.weight = torch.as_tensor(weight, device=dev, dtype=torch.float32).contiguous()
        self.cols, self.eps, self.max_rows = self.weight.shape[0], eps, max_rows
        self.act_dtype, self.out_dtype, self.scale_group = act_dtype, out_dtype, scale_group
        self.y = torch.empty(max_rows, self.cols, device=dev, dtype=out_dtype)
        self.scale = None
        if out_dtype == torch.float8_e4m3fn:
            groups = self.cols // scale_group if scale_group else 1
            self.scale = torch.empty(max_rows, groups, device=dev, dtype=torch.float32)
        self._call, self._w = B.entry("rssm_add_rmsnorm"), self.weight.data_ptr()
        self._index = _index(self.weight.device)
        self._plans = {}

    def dims(self, rows):
        return B.NormDims(rows, self.cols, self.scale_group, torch_dtype_code(self.act_dtype),
                          _code(self.out_dtype))

    def _plan(self, rows):
        """A reference to the dims of rows rows, the outputs and their addresses (no outputs
        beyond max_rows)."""
        p = self._plans.get(rows)
        if p is None:
            y = scale = None
            if rows <= self.max_rows:
                y = self.y[:rows]
                scale = None if self.scale is None else self.scale[:rows]
            p = (ctypes.byref(self.dims(rows)), y, scale, B._ptr(y), B._ptr(scale))
            if rows <= self.max_rows:
                self._plans[rows] = p
        return p

    def __call__(self, x, residual=None, residual_out=None, y=None, scale=None, stream=None):
        """Returns (y, scale) (scale None unless y is 8-bit). residual_out None: the sum
        replaces residual (without a residual it is not stored)."""
        n = x.numel()
        rows = n // self.cols
        if rows * self.cols != n or (rows > self.max_rows and
                                     (y is None or (scale is None and self.scale is not None))):
            raise ValueError("x must be [rows, %d], rows <= %d unless the outputs are given"
                             % (self.cols, self.max_rows))
        for t in (x, residual, residual_out):
            if t is not None and (t.dtype is not self.act_dtype or t.numel() != n or
                                  not t.is_contiguous() or t.get_device() != self._index):
                raise ValueError("x and the residuals: dense [rows, %d] %s on the runner's device"
                                 % (self.cols, self.act_dtype))
        dims, own_y, own_scale, y_ptr, scale_ptr = self._plan(rows)
        if y is None:
            y = own_y
        else:
            y_ptr = _check_out("y", y, n, self.out_dtype, self._index)
        if scale is None:
            scale = own_scale
        elif self.scale is not None:
            scale_ptr = _check_out("scale", scale, rows * self.scale.shape[1], torch.float32,
                                   self._index)
        res = None if residual is None else residual.data_ptr()
        rc = self._call(dims, x.data_ptr(), res, self._w, self.eps,
                        res if residual_out is None else residual_out.data_ptr(), y_ptr, scale_ptr,
                        B._stream(stream))
        if rc:
            raise B.RSSMError("rssm_add_rmsnorm", rc)
        return y, scale
