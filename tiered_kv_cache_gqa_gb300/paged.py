"""The operators around a paged KV cache on torch tensors: rope, PagedCache with append, attend, gather, and beam search:
beam_select, and PagedLayers with reorder.

Thin wrappers: they check the arguments, allocate outputs with torch's allocator on the current stream of the tensors'
device, and call the C functions of the same names (include/tkv.h), which say what is computed and what a kernel does
with positions, pages and lengths that make no sense.  An attention's workspace (12 to 23 MB at d 128) is kept by the
thread for its next attentions on that stream.  Everything runs on torch's current stream; nothing synchronises, and
every call can be captured into a CUDA graph.

    table  = rope_table(max_positions, 128)
    rotary = Rotary(table)
    cache  = PagedCache.empty(num_pages, page_table, lengths, num_kv_heads=8, head_dim=128, page_size=64)
    lengths += n                                              # the step's tokens count
    q = rope(q, rotary, positions)                            # [rows, Hq, d]
    cache.append(k, v, cu_tokens, rotary=rotary, positions=positions)
    out = cache.attend(q, cu_tokens)

and with beams, the batch being groups * beams sequences:

    layers = PagedLayers(caches)                              # of all layers; one page table, one lengths
    scores, beams, tokens = beam_select(logits, scores)       # logits [groups, beams, vocab]
    layers.reorder(beams)                                     # each sequence goes on from the beam that it was given
"""
import math
import threading

from . import (CUDA_STREAM_LEGACY, TKV_BF16, TKV_EINVAL, TKV_FP16, TKV_FP32, TKV_INT4, TKV_E4M3, TKV_OK, PagedDesc, RotaryDesc, TkvError,
               load)

_torch = _raw_stream = _current_device = _capturing = _int32 = _grad_enabled = _written = _turn = None
_DTYPES = {}
_RECORDS = {18 * 64: (TKV_INT4, 64), 18 * 128: (TKV_INT4, 128), 32 * 64 + 16: (TKV_E4M3, 64), 32 * 128 + 16: (TKV_E4M3, 128)}
_select_sizes = {}   # workspaces of beam_select, by device and shape
_own = threading.local()   # .work: the thread's workspaces of the attention, by device and stream


def _types():
    """torch, imported at the first use (the package itself does not need it)."""
    global _torch, _raw_stream, _current_device, _capturing, _int32, _grad_enabled, _written, _turn
    if _torch is None:
        import torch
        _DTYPES.update({torch.bfloat16: TKV_BF16, torch.float16: TKV_FP16, torch.float32: TKV_FP32})
        _int32 = torch.int32
        # the handle of a device's current stream and the current device, without an object around them
        _raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        _capturing = torch._C._cuda_isCurrentStreamCapturing
        # of tensors that a kernel writes for the caller: autograd notices if it had kept them for a backward pass
        _grad_enabled, _written = torch.is_grad_enabled, torch.autograd.graph.increment_version

        class Turn(torch.autograd.Function):
            @staticmethod
            def forward(ctx, to, x, rotary, positions, inverse, status):
                """Turns x into `to` (a new tensor if None), or `to` in place if x is None.  What is written comes first:
                where it is a view, autograd takes the first gradient for what the view held before."""
                y = _rope(to if x is None else x, rotary, positions, to, inverse, status)
                ctx.rotary, ctx.inverse, ctx.in_place = rotary, inverse, x is None
                ctx.save_for_backward(positions, rotary.table)   # a change of either before the backward pass is an error
                if to is not None:
                    ctx.mark_dirty(y)
                return y

            @staticmethod
            def backward(ctx, grad):
                positions, _ = ctx.saved_tensors
                before = None
                if not ctx.in_place and ctx.needs_input_grad[0]:
                    # what `to` held does not matter; a zero and not None, or what surrounds a view would get no gradient
                    before = _torch.zeros_like(grad)
                if ctx.needs_input_grad[0 if ctx.in_place else 1]:
                    grad = grad if grad.shape[2] <= 1 or grad.stride(2) == 1 else grad.contiguous()
                    grad = rope(grad, ctx.rotary, positions, inverse=not ctx.inverse)
                else:
                    grad = None
                return (grad, None) + (None,) * 4 if ctx.in_place else (before, grad) + (None,) * 4

        _turn = Turn.apply
        _torch = torch
    return _torch


def _refuse(where, why):
    e = TkvError(TKV_EINVAL, where)
    e.args = ("%s: %s" % (e.args[0], why),)
    raise e


# What follows runs at every call, in front of kernels of a few microseconds.  An entry point looks at all that matters in one
# condition; where it does not hold, the checks below say what is wrong.
def _on(x, where, what, dtype=None, dim=None, device=None):
    """x is a CUDA tensor, of that type and dimension, on that device."""
    if not isinstance(x, _torch.Tensor) or not x.is_cuda:
        _refuse(where, "%s is not a CUDA tensor" % what)
    if dtype is not None and x.dtype != dtype:
        _refuse(where, "%s is %s, not %s" % (what, x.dtype, dtype))
    if dim is not None and x.dim() != dim:
        _refuse(where, "%s has %d dimensions, not %s" % (what, x.dim(), dim))
    if device is not None and x.get_device() != device.index:
        _refuse(where, "%s is on %s, not on %s" % (what, x.device, device))


def _is_int32(x, where, what, shape, device):
    """x is a contiguous int32 tensor of that shape."""
    if isinstance(x, _torch.Tensor) and x.dtype is _int32 and x.shape == shape and x.is_cuda and x.get_device() == device.index and x.is_contiguous():
        return
    _on(x, where, what, _int32, None, device)
    if x.shape != shape or not x.is_contiguous():
        _refuse(where, "%s has to be a contiguous int32 tensor %s, not %s" % (what, list(shape), list(x.shape)))


def _call(fn, where, device, *args):
    """The C call on the tensors' device (its index), behind what its current stream holds."""
    if _current_device() != device:
        with _torch.cuda.device(device):
            rc = fn(*args, _raw_stream(device) or CUDA_STREAM_LEGACY)
    else:
        rc = fn(*args, _raw_stream(device) or CUDA_STREAM_LEGACY)
    if rc != TKV_OK:
        raise TkvError(rc, where)


def _workspace(size, index, device):
    """`size` bytes for kernels that are enqueued next on the device's current stream, kept by the thread or, in a capture, new."""
    if _current_device() != index or _capturing():
        return _torch.empty(size, dtype=_torch.uint8, device=device)
    try:
        kept = _own.work
    except AttributeError:
        kept = _own.work = {}
    key = index, _raw_stream(index)
    work = kept.get(key)
    if work is None or work.numel() < size:
        work = kept[key] = _torch.empty(size, dtype=_torch.uint8, device=device)
    return work


def _status_ptr(status, where, device):
    if status is None:
        return None
    _on(status, where, "status", _int32, None, device)
    if status.numel() < 1:
        _refuse(where, "status is empty")
    return status.data_ptr()


def rope_table(max_positions, rot_dim, base=10000.0, device="cuda", freq=None):
    """The cosines and sines of a rotation, fp32 [max_positions, rot_dim / 2, 2], computed in 64 bits.

    Pair j turns by position * base ** (-2 j / rot_dim), or by position * freq[j] (a list or tensor of rot_dim / 2
    numbers: scaled or repeated ladders)."""
    torch = _types()
    pairs = rot_dim // 2
    if rot_dim < 2 or rot_dim % 2 or max_positions < 1:
        _refuse("rope_table", "rot_dim is %s, max_positions %s: an even number, at least 1" % (rot_dim, max_positions))
    if freq is None:
        freq = float(base) ** (-torch.arange(pairs, dtype=torch.float64, device=device) / pairs)
    else:
        freq = torch.as_tensor(freq, dtype=torch.float64, device=device)
        if freq.shape != (pairs,):
            _refuse("rope_table", "freq is %s, not one number a pair" % list(freq.shape))
    angle = torch.arange(max_positions, dtype=torch.float64, device=device)[:, None] * freq
    return torch.stack([angle.cos(), angle.sin()], dim=-1).float().contiguous()


class Rotary:
    """A rotation of positions: the table, and which axis each pair of channels follows.

    pair_axis: the axis of each pair (0 for all if None), e.g. [0] * 16 + [1] * 24 + [2] * 24 for sections of
    time, height and width.  interleaved: pair j is channels (2 j, 2 j + 1), not (j, j + pairs)."""

    def __init__(self, table, pair_axis=None, interleaved=False):
        torch, w = _types(), "Rotary"
        _on(table, w, "table", torch.float32, 3)
        if not table.is_contiguous() or table.shape[2] != 2 or table.shape[0] < 1 or not 1 <= table.shape[1] <= 256:
            _refuse(w, "table is contiguous [max_positions, pairs <= 256, 2], not %s" % list(table.shape))
        axes = [0] * table.shape[1] if pair_axis is None else [int(x) for x in pair_axis]
        if len(axes) != table.shape[1] or not all(0 <= x < 4 for x in axes):
            _refuse(w, "pair_axis has an axis 0 .. 3 for each pair")
        self.table, self.num_axes, self.pairs = table, max(axes) + 1, table.shape[1]
        self.device, self._index = table.device, table.get_device()
        d = self._first = RotaryDesc()
        d.table, d.max_positions, d.pairs = table.data_ptr(), table.shape[0], table.shape[1]
        d.num_axes, d.interleaved = self.num_axes, int(bool(interleaved))
        d.pair_axis[:len(axes)] = axes
        self._own = threading.local()

    def _desc(self, positions, rows, where, inverse=False):
        """The calling thread's descriptor, with these positions: the C call has read it when it returns."""
        try:
            d = self._own.desc
        except AttributeError:
            d = self._own.desc = RotaryDesc.from_buffer_copy(self._first)
        d.inverse = inverse
        if positions is None:
            if self.num_axes > 1:
                _refuse(where, "positions are needed with %d axes" % self.num_axes)
            d.positions = None
            return d
        if not (isinstance(positions, _torch.Tensor) and positions.dtype is _int32 and positions.is_cuda and positions.get_device() == self._index):
            _on(positions, where, "positions", _int32, None, self.device)
        shape, strides = positions.shape, positions.stride()
        if len(shape) == 1:
            ok, axis_stride = shape[0] == rows and self.num_axes == 1, rows
        else:
            ok = len(shape) == 2 and shape[0] >= self.num_axes and shape[1] == rows
            axis_stride = strides[0] if ok else 0
        if not ok or (rows > 1 and strides[-1] != 1):
            _refuse(where, "positions are int32 [%d, %d], rows next to one another, not %s" % (self.num_axes, rows, list(shape)))
        d.positions, d.axis_stride = positions.data_ptr(), axis_stride
        return d


def rope(x, rotary, positions, out=None, inverse=False, status=None):
    """x [rows, heads, head_dim] (bf16, fp16 or fp32, channels contiguous) with its first 2 * pairs channels rotated.

    positions: int32 [rows] or [axes, rows].  out: a tensor like x that does not overlap it, or x itself; a new one if None.
    inverse=True turns back.  Autograd differentiates the call, with respect to x and any number of times: the gradient is
    rope(grad, ..., inverse=not inverse).  As with torch's own operators, a backward pass that is captured into a CUDA graph
    wants its forward pass captured with it, and leaves of which no eager graph is alive."""
    _types()
    if x is not None and _grad_enabled() and (getattr(x, "requires_grad", False) or getattr(out, "requires_grad", False)):
        return _turn(out, None if out is x else x, rotary, positions, inverse, status)
    y = _rope(x, rotary, positions, out, inverse, status)
    if out is not None:
        _written(out)
    return y


def _rope(x, rotary, positions, out, inverse, status):
    w, torch = "rope", _torch
    _on(x, w, "x", None, 3)
    dt = _DTYPES.get(x.dtype)
    if dt is None:
        _refuse(w, "x is %s: bf16, fp16 or fp32" % x.dtype)
    if not isinstance(rotary, Rotary) or rotary._index != x.get_device():
        _refuse(w, "rotary is not a Rotary on %s" % x.device)
    if positions is None:
        _refuse(w, "positions are needed")
    shape, xs = x.shape, x.stride()
    rows, heads, d = shape
    if out is None:
        out = torch.empty(shape, dtype=x.dtype, device=rotary.device)
    elif out is not x:
        _on(out, w, "out", x.dtype, 3, rotary.device)
        if out.shape != shape:
            _refuse(w, "out is %s, x is %s" % (list(out.shape), list(shape)))
    os_ = out.stride()
    if rows and d > 1 and (xs[2] != 1 or os_[2] != 1):
        _refuse(w, "the channels of x and out have to be contiguous")
    desc = rotary._desc(positions, rows, w, inverse)
    if rows:
        _call(load().tkv_rope, w, rotary._index, desc, x.data_ptr(), out.data_ptr(), dt, rows, heads, d, xs[0], xs[1], os_[0],
              os_[1], _status_ptr(status, w, rotary.device))
    return out


class PagedCache:
    """A paged cache in the caller's tensors; keeps them alive, writes nothing but pages (PagedLayers.reorder the page table too).

    pages       bf16 or fp16 [num_pages, Hkv, 2, page_size, d], or uint8 [num_pages, Hkv, page_size / 16, 18 d]: 4 bits,
                [..., 32 d + 16]: 8 bits, E4M3 with a power of two for each block of 16 positions and head, which never falls while
                the block lives: drafted rows that are taken back leave theirs behind
    page_table  int32 [batch, max_pages]: position p of sequence b lies in page page_table[b, p // page_size]
    lengths     int32 [batch]: positions of each sequence, the step's own included; read by every call, on the device
    k_gain, v_gain  fp32 [Hkv] > 0, 4 bits only: a value is code * scale * gain (1 if None)

    A step is ragged: rows cu_tokens[b] .. cu_tokens[b + 1] of k, v, q are the last positions of sequence b (cu_tokens
    int32 [batch + 1]).  `status` (an int32 tensor that the caller clears) is raised where a row or page has no place, or a
    kernel's wait ran out; without it nothing reports what the device finds wrong.  The calls have no gradients: their results
    are not part of autograd's graphs, whatever k, v and q are."""

    def __init__(self, pages, page_table, lengths, k_gain=None, v_gain=None):
        torch, w = _types(), "PagedCache"
        _on(pages, w, "pages")
        if not pages.is_contiguous() or pages.numel() == 0:
            _refuse(w, "pages is not contiguous, or empty")
        c = PagedDesc()
        if pages.dtype == torch.uint8:
            found = _RECORDS.get(pages.shape[3]) if pages.dim() == 4 else None
            if found is None:
                _refuse(w, "4-bit pages are [num_pages, Hkv, page_size / 16, 18 d], 8-bit ones [..., 32 d + 16], d 64 or 128, not %s" % list(pages.shape))
            (c.kv_type, c.head_dim), c.page_size = found, pages.shape[2] * 16
            if c.kv_type == TKV_E4M3 and (k_gain is not None or v_gain is not None):
                _refuse(w, "gains belong to 4-bit pages")
        else:
            if pages.dtype not in (torch.bfloat16, torch.float16) or pages.dim() != 5 or pages.shape[2] != 2:
                _refuse(w, "16-bit pages are bf16 or fp16 [num_pages, Hkv, 2, page_size, d], not %s %s" % (pages.dtype, list(pages.shape)))
            if k_gain is not None or v_gain is not None:
                _refuse(w, "gains belong to 4-bit pages")
            c.kv_type, c.head_dim, c.page_size = _DTYPES[pages.dtype], pages.shape[4], pages.shape[3]
        if c.head_dim not in (64, 128):
            _refuse(w, "head_dim is %d: 64 or 128" % c.head_dim)
        if not 16 <= c.page_size <= 65536 or c.page_size & (c.page_size - 1):
            _refuse(w, "page_size is %d: a power of two, 16 .. 65536" % c.page_size)
        _on(page_table, w, "page_table", torch.int32, 2, pages.device)
        if not page_table.is_contiguous() or page_table.numel() == 0:
            _refuse(w, "page_table is not contiguous, or empty")
        _is_int32(lengths, w, "lengths", (page_table.shape[0],), pages.device)
        if page_table.shape[1] * c.page_size > 1 << 30:
            _refuse(w, "a sequence has at most 2^30 positions")
        for name, g in (("k_gain", k_gain), ("v_gain", v_gain)):
            if g is not None:
                _on(g, w, name, torch.float32, 1, pages.device)
                if g.shape[0] != pages.shape[1] or not g.is_contiguous():
                    _refuse(w, "%s has one number a KV head" % name)
        c.pages, c.page_table, c.lengths = pages.data_ptr(), page_table.data_ptr(), lengths.data_ptr()
        c.k_gain = None if k_gain is None else k_gain.data_ptr()
        c.v_gain = None if v_gain is None else v_gain.data_ptr()
        c.num_pages, c.num_kv_heads = pages.shape[0], pages.shape[1]
        c.batch, c.max_pages = page_table.shape
        self.pages, self.page_table, self.lengths, self.k_gain, self.v_gain = pages, page_table, lengths, k_gain, v_gain
        self.device, self.num_kv_heads, self.head_dim, self.page_size = pages.device, c.num_kv_heads, c.head_dim, c.page_size
        self.batch, self.max_pages, self.is_int4 = c.batch, c.max_pages, c.kv_type == TKV_INT4
        self._any16 = c.kv_type in (TKV_INT4, TKV_E4M3)   # pages that take rows of either 16-bit type
        # what each call reads of the descriptor, without a ctypes access
        self._c, self._kv_type, self._cu_shape, self._index = c, c.kv_type, (c.batch + 1,), pages.get_device()
        self._sizes = {}   # of workspaces

    @classmethod
    def empty(cls, num_pages, page_table, lengths, *, num_kv_heads, head_dim, page_size, dtype="int4", k_gain=None, v_gain=None):
        """A cache with new pages on the page table's device; dtype "int4", "e4m3", torch.bfloat16 or torch.float16."""
        torch = _types()
        if dtype == "int4" or dtype == "e4m3":
            record = 18 * head_dim if dtype == "int4" else 32 * head_dim + 16
            pages = torch.zeros(num_pages, num_kv_heads, page_size // 16, record, dtype=torch.uint8, device=page_table.device)
        else:
            pages = torch.zeros(num_pages, num_kv_heads, 2, page_size, head_dim, dtype=dtype, device=page_table.device)
        return cls(pages, page_table, lengths, k_gain, v_gain)

    def _rows(self, x, where, what, heads):
        """x [rows, heads, d] of a 16-bit type that fits the pages, 16-byte pieces; its element type."""
        dt = _DTYPES.get(x.dtype) if isinstance(x, _torch.Tensor) else None
        if dt == self._kv_type or (self._any16 and (dt == TKV_BF16 or dt == TKV_FP16)):
            shape, s = x.shape, x.stride()
            if (len(shape) == 3 and shape[2] == self.head_dim and (heads is None or shape[1] == heads) and s[2] == 1 and
                    not (s[0] | s[1]) % 8 and not x.data_ptr() % 16 and x.get_device() == self._index and x.is_cuda):
                return dt
        _on(x, where, what, None, 3, self.device)
        dt = _DTYPES.get(x.dtype)
        if dt == TKV_FP32 or dt is None or (not self._any16 and dt != self._kv_type):
            _refuse(where, "%s is %s, the pages are %s" % (what, x.dtype, self.pages.dtype))
        if x.shape[2] != self.head_dim or (heads is not None and x.shape[1] != heads):
            _refuse(where, "%s is %s, not [rows, %s, %d]" % (what, list(x.shape), heads or "Hq", self.head_dim))
        self._pieces(x, where, what)
        return dt

    def _pieces(self, x, where, what):
        s = x.stride()
        e = 16 // x.element_size()
        if s[2] != 1 or s[0] % e or s[1] % e or x.data_ptr() % 16:
            _refuse(where, "%s has to lie in 16-byte pieces: contiguous channels, aligned rows and heads" % what)

    def _work(self, hq, max_new):
        """A workspace for an attention that is enqueued next on the current stream.

        A thread keeps one a stream, for all its caches: what it enqueues there runs in order.  Other threads' launches may
        come between the two of a call, so they have their own; so has a call that is captured, which may run beside any
        other later."""
        size = self._sizes.get((hq, max_new))
        if size is None:
            with _torch.cuda.device(self._index):
                size = self._sizes[hq, max_new] = load().tkv_paged_attention_workspace(self._c, hq, max_new)
        return _workspace(size, self._index, self.device)

    def append(self, k, v, cu_tokens, rotary=None, positions=None, status=None):
        """Writes k, v [rows, Hkv, d] (bf16 or fp16) to their places, k rotated on the way if `rotary` is given:
        by positions (int32 [rows] or [axes, rows]), or by the places in the cache if None."""
        w = "append"
        dt = self._rows(k, w, "k", self.num_kv_heads)
        rows = k.shape[0]
        if self._rows(v, w, "v", self.num_kv_heads) != dt or v.shape[0] != rows:
            _refuse(w, "v is not like k")
        _is_int32(cu_tokens, w, "cu_tokens", self._cu_shape, self.device)
        desc = None
        if rotary is not None:
            if not isinstance(rotary, Rotary) or rotary.device != self.device:
                _refuse(w, "rotary is not a Rotary on %s" % self.device)
            if 2 * rotary.pairs > self.head_dim:
                _refuse(w, "rotary turns %d channels of %d" % (2 * rotary.pairs, self.head_dim))
            desc = rotary._desc(positions, rows, w)
        elif positions is not None:
            _refuse(w, "positions without rotary")
        if rows:
            ks, vs = k.stride(), v.stride()
            _call(load().tkv_paged_append, w, self._index, self._c, desc, k.data_ptr(), v.data_ptr(), dt, rows, ks[0], ks[1],
                  vs[0], vs[1], cu_tokens.data_ptr(), _status_ptr(status, w, self.device))

    def gather(self, cu_tokens, rows, dtype=None, k=None, v=None, lengths=None, status=None):
        """Reads positions back: k, v [rows, Hkv, d] of dtype (bf16 if None; fp16, fp32), addressed like an append.

        rows: the extent of the outputs, cu_tokens[batch] at least (rows behind it are left as they were).
        lengths: the ends of the ranges (the cache's own lengths if None).  k, v: tensors to write to."""
        w = "gather"
        torch = _types()
        _is_int32(cu_tokens, w, "cu_tokens", self._cu_shape, self.device)
        shape = (int(rows), self.num_kv_heads, self.head_dim)
        if rows < 0 or (k is None) != (v is None):
            _refuse(w, "rows is at least 0; k and v come together")
        if k is None:
            dtype = torch.bfloat16 if dtype is None else dtype
            if dtype not in _DTYPES:
                _refuse(w, "dtype is %s: bf16, fp16 or fp32" % dtype)
            k = torch.empty(shape, dtype=dtype, device=self.device)
            v = torch.empty(shape, dtype=dtype, device=self.device)
        else:
            for name, x in (("k", k), ("v", v)):
                _on(x, w, name, k.dtype if dtype is None else dtype, 3, self.device)
                if x.shape != shape or x.dtype not in _DTYPES:
                    _refuse(w, "%s is not bf16, fp16 or fp32 %s" % (name, list(shape)))
                self._pieces(x, w, name)
            _written((k, v))
        c = self._c
        if lengths is not None:
            _is_int32(lengths, w, "lengths", (self.batch,), self.device)
            c = PagedDesc.from_buffer_copy(c)
            c.lengths = lengths.data_ptr()
        if rows:
            ks, vs = k.stride(), v.stride()
            _call(load().tkv_paged_gather, w, self._index, c, k.data_ptr(), v.data_ptr(), _DTYPES[k.dtype], rows, ks[0], ks[1],
                  vs[0], vs[1], cu_tokens.data_ptr(), _status_ptr(status, w, self.device))
        return k, v

    def attend(self, q, cu_tokens, max_new=None, max_len=None, window=0, scale=None, out=None, return_lse=False, lse=None,
               status=None):
        """Attention of the step's queries q [rows, Hq, d] over the cache: out like q, and with return_lse (out, lse
        fp32 [rows, Hq]).  A query sees the positions up to its own and, with window > 0, the last `window` of them.

        max_new, max_len: the host's estimates of the most queries and positions of a sequence (they choose the split of
        the work, not the result); the rows a sequence at least, and the table's whole extent, if None.
        scale: 1 / sqrt(d) if None.  out, lse: tensors to write to (rows behind cu_tokens[batch] stay as they were)."""
        w = "attend"
        torch = _types()
        dt = self._rows(q, w, "q", None)
        shape = q.shape
        rows, hq, d = shape
        if hq < 1 or hq % self.num_kv_heads:
            _refuse(w, "%d query heads over %d KV heads" % (hq, self.num_kv_heads))
        _is_int32(cu_tokens, w, "cu_tokens", self._cu_shape, self.device)
        max_new = max(1, -(-rows // self.batch)) if max_new is None else int(max_new)
        max_len = self.max_pages * self.page_size if max_len is None else int(max_len)
        window = int(window)
        if not 1 <= max_new < 1 << 31 or not 0 <= window < 1 << 31:
            _refuse(w, "max_new is %d, window %d: int32, at least 1 and 0" % (max_new, window))
        max_len = min(max(1, max_len), (1 << 31) - 1)
        scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
        if out is None:
            out = torch.empty(shape, dtype=q.dtype, device=self.device)
        else:
            _on(out, w, "out", q.dtype, 3, self.device)
            if out.shape != shape:
                _refuse(w, "out is %s, q is %s" % (list(out.shape), list(shape)))
            self._pieces(out, w, "out")
            _written(out)
        if lse is not None:
            _on(lse, w, "lse", torch.float32, 2, self.device)
            if lse.shape != (rows, hq) or not lse.is_contiguous():
                _refuse(w, "lse is a contiguous [%d, %d]" % (rows, hq))
            _written(lse)
        elif return_lse:
            lse = torch.empty((rows, hq), dtype=torch.float32, device=self.device)
        if rows:
            work = self._work(hq, max_new)
            qs, os_ = q.stride(), out.stride()
            _call(load().tkv_paged_attention, w, self._index, self._c, q.data_ptr(), out.data_ptr(),
                  None if lse is None else lse.data_ptr(), dt, rows, hq, qs[0], qs[1], os_[0], os_[1], cu_tokens.data_ptr(),
                  max_new, max_len, window, scale, work.data_ptr(), work.numel(), _status_ptr(status, w, self.device))
        return (out, lse) if return_lse else out


class PagedLayers:
    """The caches of a model's layers, which share a page table and lengths, each with pages of its own; keeps them alive.

    Sequences come in groups of beams: sequence g * beams + w is beam w of group g."""

    def __init__(self, caches):
        _types()
        w, caches = "PagedLayers", list(caches)
        if not caches or not all(isinstance(c, PagedCache) for c in caches):
            _refuse(w, "caches is a list of PagedCache, not empty")
        first = caches[0]
        for c in caches:
            if c.page_table is not first.page_table and c.page_table.data_ptr() != first.page_table.data_ptr():
                _refuse(w, "the caches have to share one page table")
            if c.lengths is not first.lengths and c.lengths.data_ptr() != first.lengths.data_ptr():
                _refuse(w, "the caches have to share one lengths")
            if (c.batch, c.max_pages, c.page_size, c._index) != (first.batch, first.max_pages, first.page_size, first._index):
                _refuse(w, "the caches differ in batch, pages a sequence, page size or device")
        if first.pages.numel() and len({c.pages.data_ptr() for c in caches}) != len(caches):
            _refuse(w, "two caches have the same pages")
        self.caches, self.batch, self.device, self._index = caches, first.batch, first.device, first._index
        self._c = (PagedDesc * len(caches))(*(c._c for c in caches))

    def reorder(self, parents, status=None):
        """Sequence g * beams + w goes on from g * beams + parents[g, w]; parents int32 [groups, beams], as beam_select gives
        `beams`; a negative one keeps what the sequence has.

        The page table's columns before the current page (lengths // page_size) become the parent's; what the current page holds
        is copied in all layers.  The pages from the current one on have to be each sequence's own, those before may be
        shared.  To hand a prompt that sequence w has appended to its group: parents of w, with the lengths of all set."""
        w = "reorder"
        if not (isinstance(parents, _torch.Tensor) and parents.dtype is _int32 and parents.is_cuda and parents.get_device() == self._index):
            _on(parents, w, "parents", _int32, 2, self.device)
        shape = parents.shape
        if len(shape) != 2 or shape[0] * shape[1] != self.batch or not parents.is_contiguous():
            _refuse(w, "parents are contiguous int32 [groups, beams], %d sequences, not %s" % (self.batch, list(shape)))
        if not 1 <= shape[1] <= 32:
            _refuse(w, "%d beams: 1 to 32" % shape[1])
        _call(load().tkv_paged_reorder, w, self._index, self._c, len(self.caches), parents.data_ptr(), shape[1],
              _status_ptr(status, w, self.device))


def beam_select(logits, scores, count=None, finished=None, eos=None):
    """The best `count` (the number of beams if None) continuations of each sequence: (scores fp32, beams int32, tokens int32), each
    [batch, count], in descending order, ties to the lowest beam and token.

    logits    [batch, beams, vocab] bf16, fp16 or fp32, the vocabulary contiguous: any strides and alignment of the rows
    scores    fp32 [batch, beams]: sums of log probabilities so far; -inf takes a beam out
    finished  bool or uint8 [batch, beams]: such a beam offers token `eos` with its own score, and nothing else
    A candidate's score is scores + log_softmax(logits); where there are fewer than `count`, score -inf, beam -1, token -1.
    Up to 64 beams, of which PagedLayers.reorder follows 32.  The call has no gradient."""
    w, torch = "beam_select", _types()
    if not (isinstance(logits, torch.Tensor) and logits.is_cuda and logits.dim() == 3):
        _on(logits, w, "logits", None, 3)
    dt = _DTYPES.get(logits.dtype)
    if dt is None:
        _refuse(w, "logits is %s: bf16, fp16 or fp32" % logits.dtype)
    shape, s, device = logits.shape, logits.stride(), logits.device
    batch, beams, vocab = shape
    index = device.index
    count = beams if count is None else int(count)
    if not (1 <= beams <= 64 and 1 <= count <= 64 and vocab >= 1 and beams * vocab <= 0x7FFFFF00 and batch * beams <= 0x7FFFFFFF // 64):
        _refuse(w, "%s logits, count %d: beams and count are 1 to 64, beams * vocab is below 2^31 - 256" % (list(shape), count))
    if s[2] != 1 and vocab > 1:
        _refuse(w, "the vocabulary has to be contiguous")
    if not (isinstance(scores, torch.Tensor) and scores.dtype is torch.float32 and scores.is_cuda and scores.get_device() == index):
        _on(scores, w, "scores", torch.float32, 2, device)
    if scores.shape != shape[:2] or not scores.is_contiguous():
        _refuse(w, "scores is a contiguous [%d, %d]" % (batch, beams))
    done, last = None, 0
    if finished is not None:
        _on(finished, w, "finished", None, 2, device)
        if finished.dtype not in (torch.bool, torch.uint8) or finished.shape != shape[:2] or not finished.is_contiguous():
            _refuse(w, "finished is a contiguous bool or uint8 [%d, %d]" % (batch, beams))
        if eos is None or not 0 <= int(eos) < vocab:
            _refuse(w, "eos is %s: a token of the vocabulary" % eos)
        done, last = finished.data_ptr(), int(eos)
    empty, size = torch.empty, (batch, count)
    out, out_beams, tokens = empty(size, dtype=torch.float32, device=device), empty(size, dtype=_int32, device=device), empty(size, dtype=_int32, device=device)
    if batch:
        key = index, dt, batch, beams, vocab, count
        size = _select_sizes.get(key)
        if size is None:
            with torch.cuda.device(index):
                size = _select_sizes[key] = load().tkv_beam_select_workspace(dt, batch, beams, vocab, count)
        work = _workspace(size, index, device)
        _call(load().tkv_beam_select, w, index, logits.data_ptr(), dt, batch, beams, vocab, s[0], s[1], scores.data_ptr(), done, last, count,
              out.data_ptr(), out_beams.data_ptr(), tokens.data_ptr(), work.data_ptr(), work.numel())
    return out, out_beams, tokens
