"""Serving many requests from one paged key/value cache: block tables and slots built on the GPU
(fa_kv_reserve, fa_kv_release), rotary position embedding with several axes (fa_rope, and
fa_rope_append, which also writes the cache) and attention over the cache (fa_paged_fwd).
PagedKV keeps the state of such a cache and runs the four in order.

As in the rest of the binding, the functions marshal arguments into the C ABI of
``include/fa.h``; all lengths, tables and counts stay on the device, no call synchronises, and
everything can be captured in a CUDA graph when the output buffers are given."""
from __future__ import annotations

import ctypes
import math

__all__ = ["RopeTable", "PagedKV", "fa_kv_reserve", "fa_kv_release", "fa_rope", "fa_rope_append", "fa_paged_fwd",
           "paged_workspace_bytes"]


class _RopeSpec(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("num_axes", ctypes.c_int),
                ("inv_freq", ctypes.POINTER(ctypes.c_double)), ("axis", ctypes.POINTER(ctypes.c_int))]


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("block_stride", ctypes.c_longlong),
                ("slot_stride", ctypes.c_longlong), ("head_stride", ctypes.c_longlong), ("num_blocks", ctypes.c_int),
                ("page_size", ctypes.c_int), ("Hkv", ctypes.c_int), ("d", ctypes.c_int)]


def declare(L) -> None:
    """Argument types of the paged-cache entry points of the loaded library."""
    vp, ci, ll, cf = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float
    L.fa_kv_reserve.argtypes = [vp, vp, ci, vp, ll, ci, vp, vp, ci, ci, ci, vp, vp, vp, vp, vp, vp]
    L.fa_kv_release.argtypes = [vp, vp, ci, vp, ll, ci, vp, vp, ci, ci, vp, vp, vp]
    rope = [vp, ll, vp, ll, ci, vp, ll, vp, ll, ci, ci, ci, vp, ll, ctypes.POINTER(_RopeSpec), ci, vp]
    append = [vp, ll, vp, ll, ci, vp, ll, vp, ll, ci, vp, ll, ctypes.POINTER(_RopeSpec), ctypes.POINTER(_Cache), vp, vp]
    paged = [vp, ll, ctypes.POINTER(_Cache), vp, ll, ci, vp, vp, ci, ci, ci, ci, cf, ci, ci, vp, vp, vp, ctypes.c_size_t, vp]
    for name, args in (("fa_rope", rope), ("fa_rope_append", append), ("fa_paged_fwd", paged)):
        for f16 in ("", "_f16"):
            getattr(L, name + f16).argtypes = args
            getattr(L, name + f16).restype = ci
    L.fa_kv_reserve.restype = L.fa_kv_release.restype = ci
    L.fa_paged_workspace_bytes.argtypes = [ci, ci, ci]
    L.fa_paged_workspace_bytes.restype = ctypes.c_size_t


class _Types:
    """torch's types and stream query, looked up at the first call (the module imports without torch)."""
    ready = False


def _init() -> None:
    import torch

    import exact_attention_146_b200 as fa
    _Types.i32, _Types.i64, _Types.f32 = torch.int32, torch.int64, torch.float32
    _Types.half = {torch.bfloat16: "", torch.float16: "_f16"}
    _Types.torch, _Types.fa = torch, fa
    # the current stream's handle without building a Stream object (3 us a call)
    raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), torch.cuda.current_device
    _Types.current = (lambda: raw(device())) if raw else (lambda: torch.cuda.current_stream().cuda_stream)
    L = fa.lib()
    _Types.call = {n: getattr(L, n) for n in ("fa_kv_reserve", "fa_kv_release", "fa_rope", "fa_rope_f16", "fa_rope_append",
                                              "fa_rope_append_f16", "fa_paged_fwd", "fa_paged_fwd_f16")}
    _Types.ready = True


def _run(name, stream, *args):
    rc = _Types.call[name](*args, _Types.current() if stream is None else _Types.fa._stream_handle(stream))
    if rc != 0:
        raise _Types.fa.FaError(rc, name)


def _empty(shape, dtype, device, stream):
    """A buffer made here for a call on `stream` (None: the current one)."""
    torch = _Types.torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):   # so that its memory is not handed out again before that stream is done with it
        return torch.empty(shape, dtype=dtype, device=device)


def _like(t, shape, stream):
    """An uninitialised buffer of t's type on its device."""
    return t.new_empty(shape) if stream is None else _empty(shape, t.dtype, t.device, stream)


def _ints(name, t, n, dtype=None):
    """The pointer of a contiguous 1-D CUDA tensor of n int32 (or dtype)."""
    dtype = dtype or _Types.i32
    if t.dtype is not dtype or not t.is_cuda or t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor ({n},), got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def _table(t, R, written=False):
    """(pointer, entries from row to row, entries a row) of a block table.  One that is only read may be a
    single row for all requests (expanded: 0 entries from row to row); other rows may not overlap."""
    if t.dtype is _Types.i32 and t.is_cuda and t.dim() == 2:
        rows, width = t.shape
        if rows == R and (width <= 1 or t.stride(1) == 1):
            step = t.stride(0) if R > 1 else width
            if step < width and (step != 0 or written):
                raise ValueError(f"the rows of block_table overlap: {width} entries, {step} from row to row")
            return t.data_ptr(), step, width
    raise ValueError(f"block_table must be an int32 CUDA tensor [{R}, max_blocks] with adjacent entries, got {t.dtype} {tuple(t.shape)}")


def _rows(name, t, dtype, shape=None):
    """A [T, heads, d] tensor whose heads lie next to each other: (pointer, elements from token to token)."""
    if t.dtype is not dtype or not t.is_cuda or t.dim() != 3 or (shape is not None and t.shape != shape):
        want = "[T, heads, d]" if shape is None else tuple(shape)
        raise ValueError(f"{name} must be a {dtype} CUDA tensor {want}, got {t.dtype} {tuple(t.shape)}")
    T, H, d = t.shape
    step, head, one = t.stride()
    if (d > 1 and one != 1) or (H > 1 and head != d):
        raise ValueError(f"{name}: the heads of a token must lie next to each other, strides {t.stride()}")
    return t.data_ptr(), (step if T > 1 else H * d)


def _cache(k, v):
    """The C description of k and v caches, logically [blocks, slots, heads, d] with any strides of the first three."""
    shape, strides = k.shape, k.stride()
    for name, t in (("k_cache", k), ("v_cache", v)):
        if not t.is_cuda or len(shape) != 4 or t.dtype is not k.dtype or (shape[3] > 1 and strides[3] != 1):
            raise ValueError(f"{name} must be a 4-D CUDA tensor [blocks, slots, heads, d] with adjacent elements, got {t.dtype} {tuple(t.shape)}")
    if shape != v.shape or strides != v.stride():
        raise ValueError(f"k_cache and v_cache must have the same shape and strides, got {tuple(shape)} {strides} and {tuple(v.shape)} {v.stride()}")
    return _Cache(k.data_ptr(), v.data_ptr(), strides[0], strides[1], strides[2], shape[0], shape[1], shape[2], shape[3])


def _half(t):
    """The suffix of the entry points for t's type."""
    if not _Types.ready:
        _init()
    if t.dtype not in _Types.half:
        raise ValueError(f"bf16 or fp16 expected, got {t.dtype}")
    return _Types.half[t.dtype]


class RopeTable:
    """Frequencies of a rotary embedding: inv_freq[i] and axis[i] of pair i (axis None: one axis);
    interleaved pairs are (2i, 2i + 1), else (i, i + rot_dim / 2)."""

    def __init__(self, inv_freq, axis=None, interleaved: bool = False):
        inv = [float(x) for x in inv_freq]
        axes = [0] * len(inv) if axis is None else [int(a) for a in axis]
        if len(axes) != len(inv):
            raise ValueError(f"{len(inv)} frequencies but {len(axes)} axes")
        if not all(math.isfinite(x) for x in inv) or any(not 0 <= a < 4 for a in axes):
            raise ValueError("frequencies must be finite, axes 0 .. 3")
        self.rot_dim = 2 * len(inv)
        self.num_axes = max(axes, default=0) + 1
        self.interleaved = bool(interleaved)
        self._specs = {}
        self._inv = (ctypes.c_double * max(1, len(inv)))(*inv)
        self._axis = (ctypes.c_int * max(1, len(inv)))(*axes)

    def _spec(self, positions, T):
        """(spec, pointer, elements from axis to axis) of positions [axes, T] or [T]; axes that share one row
        (expanded) are 0 elements apart."""
        n, step = (positions.shape[0], positions.stride(0)) if positions.dim() == 2 else (1, T)
        if positions.dtype is not _Types.i32 or not positions.is_cuda or positions.dim() not in (1, 2) or \
                positions.shape[-1] != T or (T > 1 and positions.stride(-1) != 1):
            raise ValueError(f"positions must be int32 CUDA [axes, {T}] (or [{T}]), got {positions.dtype} {tuple(positions.shape)}")
        if n < self.num_axes:
            raise ValueError(f"the table uses {self.num_axes} axes, positions has {n}")
        if n > 1 and 0 != step < T:
            raise ValueError(f"the axes of positions overlap: {T} tokens, {step} elements from axis to axis")
        spec = self._specs.get(n)
        if spec is None:
            spec = self._specs[n] = ctypes.byref(_RopeSpec(self.rot_dim, int(self.interleaved), n, self._inv, self._axis))
        return spec, positions.data_ptr(), (step if n > 1 else T)


def fa_rope(q, positions, table: RopeTable, *, k=None, inverse: bool = False, q_out=None, k_out=None, stream=None):
    """Rotary embedding of q [T, Hq, d] (and k [T, Hkv, d]) bf16 or fp16 by positions [axes, T] int32;
    inverse = True is its gradient (the opposite turn).  q and k may be slices of one projection.
    Returns (q_out, k_out), or q_out alone without k; q_out may be q and k_out k (in place)."""
    f16 = _half(q)
    dtype = q.dtype
    qp, qs = _rows("q", q, dtype)
    shape = q.shape
    T, Hq, d = shape
    if q_out is None:
        q_out = _like(q, shape, stream)
    qo, qos = _rows("q_out", q_out, dtype, shape)
    kp = ko = None
    ks = kos = Hkv = 0
    if k is not None:
        kp, ks = _rows("k", k, dtype)
        shape = k.shape
        Hkv = shape[1]
        if shape[0] != T or shape[2] != d:
            raise ValueError(f"k must be [{T}, heads, {d}], got {tuple(shape)}")
        if k_out is None:
            k_out = _like(k, shape, stream)
        ko, kos = _rows("k_out", k_out, dtype, shape)
    spec, pos, ps = table._spec(positions, T)
    _run("fa_rope" + f16, stream, qp, qs, qo, qos, Hq, kp, ks, ko, kos, Hkv, T, d, pos, ps, spec, 1 if inverse else 0)
    return q_out if k is None else (q_out, k_out)


def fa_rope_append(q, k, v, positions, table: RopeTable, k_cache, v_cache, slots, *, q_out=None, stream=None):
    """Rotates q [T, Hq, d] and k [T, Hkv, d] and writes the rotated k and v [T, Hkv, d] to slots [T]
    (int64, block * page_size + slot; negative: the row is left out) of the caches, logically
    [blocks, slots, Hkv, d].  q may be None.  Returns q_out (rows without a slot as they were)."""
    f16 = _half(k)
    dtype = k.dtype
    kp, ks = _rows("k", k, dtype)
    vp, vs = _rows("v", v, dtype, k.shape)
    T, Hkv, d = k.shape
    c = _cache(k_cache, v_cache)
    if (c.Hkv, c.d) != (Hkv, d) or k_cache.dtype is not dtype:
        raise ValueError(f"shape mismatch k{tuple(k.shape)} {dtype} cache{tuple(k_cache.shape)} {k_cache.dtype}")
    qp = qo = None
    qs = qos = Hq = 0
    if q is not None:
        qp, qs = _rows("q", q, dtype)
        shape = q.shape
        Hq = shape[1]
        if shape[0] != T or shape[2] != d:
            raise ValueError(f"q must be [{T}, heads, {d}], got {tuple(shape)}")
        if q_out is None:
            q_out = _like(q, shape, stream)
        qo, qos = _rows("q_out", q_out, dtype, shape)
    spec, pos, ps = table._spec(positions, T)
    _run("fa_rope_append" + f16, stream, qp, qs, qo, qos, Hq, kp, ks, vp, vs, T, pos, ps, spec, ctypes.byref(c),
         _ints("slots", slots, T, _Types.i64))
    return q_out if q is not None else None


def fa_kv_reserve(ctx_lens, new_lens, block_table, free_blocks, free_count, *, page_size: int, num_tokens: int | None = None,
                  cu_seqlens=None, seq_lens=None, positions=None, slots=None, free_count_out=None, stream=None):
    """Takes the blocks that R requests need for new_lens more tokens (fa_kv_reserve): fills
    block_table [R, max_blocks] and returns (cu_seqlens [R + 1], seq_lens [R], positions [T], slots [T]
    int64, free_count_out [1]).  T is given by num_tokens, or by positions or slots.  seq_lens may be
    ctx_lens and free_count_out free_count (updated in place)."""
    if not _Types.ready:
        _init()
    R = ctx_lens.numel()
    given = positions if positions is not None else slots
    if num_tokens is None and given is None:
        raise ValueError("num_tokens, or positions or slots of that length, must be given")
    T = given.numel() if num_tokens is None else int(num_tokens)
    dev, i32 = ctx_lens.device, _Types.i32
    if cu_seqlens is None:
        cu_seqlens = _empty((R + 1,), i32, dev, stream)
    if seq_lens is None:
        seq_lens = _empty((R,), i32, dev, stream)
    if positions is None:
        positions = _empty((T,), i32, dev, stream)
    if slots is None:
        slots = _empty((T,), _Types.i64, dev, stream)
    if free_count_out is None:
        free_count_out = _empty((1,), i32, dev, stream)
    table, stride, width = _table(block_table, R, written=True)
    blocks = free_blocks.numel()
    _run("fa_kv_reserve", stream, _ints("ctx_lens", ctx_lens, R), _ints("new_lens", new_lens, R), R, table, stride, width,
         _ints("free_blocks", free_blocks, blocks), _ints("free_count", free_count, 1), blocks, int(page_size), T,
         _ints("cu_seqlens", cu_seqlens, R + 1), _ints("seq_lens", seq_lens, R), _ints("positions", positions, T),
         _ints("slots", slots, T, _Types.i64), _ints("free_count_out", free_count_out, 1))
    return cu_seqlens, seq_lens, positions, slots, free_count_out


def fa_kv_release(lens, done, block_table, free_blocks, free_count, *, page_size: int, lens_out=None, free_count_out=None,
                  stream=None):
    """Gives the blocks of every request with done[r] != 0 back to the free stack (fa_kv_release);
    returns (lens_out [R], free_count_out [1]).  lens_out may be lens, free_count_out free_count."""
    if not _Types.ready:
        _init()
    R = lens.numel()
    if lens_out is None:
        lens_out = _empty((R,), _Types.i32, lens.device, stream)
    if free_count_out is None:
        free_count_out = _empty((1,), _Types.i32, lens.device, stream)
    lens_p, done_p = _ints("lens", lens, R), _ints("done", done, R)
    table, stride, width = _table(block_table, R)
    blocks = free_blocks.numel()
    _run("fa_kv_release", stream, lens_p, done_p, R, table, stride, width, _ints("free_blocks", free_blocks, blocks),
         _ints("free_count", free_count, 1), blocks, int(page_size), _ints("lens_out", lens_out, R),
         _ints("free_count_out", free_count_out, 1))
    return lens_out, free_count_out


def paged_workspace_bytes(Hq: int, Hkv: int, d: int) -> int:
    if not _Types.ready:
        _init()
    return int(_Types.fa.lib().fa_paged_workspace_bytes(int(Hq), int(Hkv), int(d)))


def fa_paged_fwd(q, k_cache, v_cache, block_table, cu_seqlens, seq_lens, *, max_new: int, causal: bool = True,
                 scale: float | None = None, window: int | None = None, out=None, lse=None, return_lse: bool = True,
                 workspace=None, stream=None):
    """Exact attention of new tokens over a paged cache (fa_paged_fwd): q [T, Hq, d] bf16 or fp16, request
    r's tokens in rows cu_seqlens[r] .. cu_seqlens[r + 1] - 1 (at most max_new of them), its seq_lens[r]
    keys (the new tokens' own among them) in the blocks block_table[r] of the caches, logically
    [blocks, slots, Hkv, d].  Returns (out [T, Hq, d], lse [Hq, T] fp32 or None); rows of no request are
    left as they are in `out` and `lse` (undefined in buffers made here)."""
    f16 = _half(q)
    dtype = q.dtype
    qp, qs = _rows("q", q, dtype)
    shape = q.shape
    T, Hq, d = shape
    c = _cache(k_cache, v_cache)
    if k_cache.dtype is not dtype or c.d != d:
        raise ValueError(f"shape mismatch q{tuple(shape)} {dtype} cache{tuple(k_cache.shape)} {k_cache.dtype}")
    R = seq_lens.numel()
    table, stride, width = _table(block_table, R)
    if out is None:
        out = _like(q, shape, stream)
    elif out.dtype is not dtype or out.shape != shape or not out.is_contiguous():
        raise ValueError(f"out must be contiguous {dtype} {tuple(shape)}, got {out.dtype} {tuple(out.shape)}")
    lse_p = None
    if not return_lse:
        lse = None
    else:
        if lse is None:
            lse = _empty((Hq, T), _Types.f32, q.device, stream)
        elif lse.dtype is not _Types.f32 or lse.shape != (Hq, T) or not lse.is_contiguous():
            raise ValueError(f"lse must be contiguous fp32 {(Hq, T)}, got {lse.dtype} {tuple(lse.shape)}")
        lse_p = lse.data_ptr()
    if window is None:
        window = 0
    elif int(window) < 1:
        raise ValueError(f"window must be at least 1, got {window}")
    if workspace is None:
        workspace = _empty((max(1, paged_workspace_bytes(Hq, c.Hkv, d)),), _Types.torch.uint8, q.device, stream)
    elif not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous CUDA tensor, got strides {workspace.stride()} on {workspace.device}")
    _run("fa_paged_fwd" + f16, stream, qp, qs, ctypes.byref(c), table, stride, width, _ints("cu_seqlens", cu_seqlens, R + 1),
         _ints("seq_lens", seq_lens, R), R, T, Hq, int(max_new), d ** -0.5 if scale is None else float(scale), 1 if causal else 0,
         int(window), out.data_ptr(), lse_p, workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out, lse


class PagedKV:
    """One layer's paged cache for up to `max_requests` requests, and a step over it: reserve() takes room
    for the new tokens, append() rotates and stores them, attend() is the attention, release() gives the
    blocks of finished requests back.  Everything is on the device; nothing synchronises.  With
    several layers, one PagedKV holds the tables and the others are made with tables=that one.

    layout "hnd" keeps a head's slots of a block together in memory, "nhd" a slot's heads."""

    def __init__(self, max_requests: int, num_blocks: int, page_size: int, Hkv: int, d: int, *, max_blocks: int | None = None,
                 dtype=None, device="cuda", layout: str = "nhd", tables: "PagedKV | None" = None):
        if not _Types.ready:
            _init()
        torch = _Types.torch
        if layout not in ("nhd", "hnd"):
            raise ValueError(f"layout must be nhd or hnd, got {layout}")
        dtype = dtype or torch.bfloat16
        shape = (num_blocks, page_size, Hkv, d) if layout == "nhd" else (num_blocks, Hkv, page_size, d)
        caches = [torch.zeros(shape, dtype=dtype, device=device) for _ in range(2)]
        self.k_cache, self.v_cache = caches if layout == "nhd" else [c.permute(0, 2, 1, 3) for c in caches]
        self.page_size, self.num_blocks, self.Hkv, self.d = page_size, num_blocks, Hkv, d
        self.tables = tables or self
        if tables is not None:
            if (tables.page_size, tables.num_blocks) != (page_size, num_blocks) or tables.seq_lens.shape[0] != max_requests:
                raise ValueError("layers that share tables have the same requests, blocks and page size")
            return
        ints = dict(dtype=torch.int32, device=device)
        self.block_table = torch.zeros((max_requests, max_blocks or num_blocks), **ints)
        self.seq_lens = torch.zeros(max_requests, **ints)
        self.free_blocks = torch.arange(num_blocks - 1, -1, -1, **ints)
        self.free_count = torch.full((1,), num_blocks, **ints)
        self.cu_seqlens = torch.zeros(max_requests + 1, **ints)
        self.positions = self.slots = None
        self._buffers = {}    # rows, a power of two -> (positions, slots)
        self._last = (None, None)

    def _rows_of(self, num_tokens: int, stream):
        """Positions and slots of a step of num_tokens rows: the start of buffers of the next power of two.  They are
        kept, and a number of rows has always the same ones, as a captured step expects; all of them together
        have about four times the most rows at most."""
        if self._last[0] is None or self._last[0].shape[0] != num_tokens:
            size = max(64, 1 << max(0, num_tokens - 1).bit_length())
            if size not in self._buffers:
                self._buffers[size] = tuple(_empty((size,), t, self.seq_lens.device, stream) for t in (_Types.i32, _Types.i64))
            self._last = tuple(b[:num_tokens] for b in self._buffers[size])
        return self._last

    def reserve(self, new_lens, num_tokens: int, *, positions=None, slots=None, stream=None):
        """Room for new_lens [max_requests] int32 more tokens, num_tokens rows in all (rows behind the last
        token are allowed: a captured step of fixed size).  Returns positions and slots: those given
        ([num_tokens] int32 and int64), or buffers of this cache, which the next reserve may fill anew."""
        if self.tables is not self:
            raise ValueError("reserve on the layer that holds the tables")
        num_tokens = int(num_tokens)
        if positions is None or slots is None:
            kept = self._rows_of(num_tokens, stream)
            positions, slots = kept[0] if positions is None else positions, kept[1] if slots is None else slots
        fa_kv_reserve(self.seq_lens, new_lens, self.block_table, self.free_blocks, self.free_count, page_size=self.page_size,
                      num_tokens=num_tokens, cu_seqlens=self.cu_seqlens, seq_lens=self.seq_lens, positions=positions, slots=slots,
                      free_count_out=self.free_count, stream=stream)
        self.positions, self.slots = positions, slots
        return positions, slots

    def append(self, q, k, v, table: RopeTable, *, positions=None, q_out=None, stream=None):
        """Rotates q and k by `positions` (default: the positions in the requests) and stores k and v."""
        t = self.tables
        if t.slots is None:
            raise ValueError("reserve before append")
        return fa_rope_append(q, k, v, t.positions if positions is None else positions, table, self.k_cache, self.v_cache, t.slots,
                              q_out=q_out, stream=stream)

    def attend(self, q, *, max_new: int, causal: bool = True, scale=None, window=None, out=None, lse=None, return_lse=True,
               workspace=None, stream=None):
        """Attention of the new tokens' (rotated) q [T, Hq, d]."""
        t = self.tables
        return fa_paged_fwd(q, self.k_cache, self.v_cache, t.block_table, t.cu_seqlens, t.seq_lens, max_new=max_new, causal=causal,
                            scale=scale, window=window, out=out, lse=lse, return_lse=return_lse, workspace=workspace, stream=stream)

    def release(self, done, *, stream=None):
        """Gives back the blocks of every request with done[r] != 0 ([max_requests] int32)."""
        if self.tables is not self:
            raise ValueError("release on the layer that holds the tables")
        fa_kv_release(self.seq_lens, done, self.block_table, self.free_blocks, self.free_count, page_size=self.page_size,
                      lens_out=self.seq_lens, free_count_out=self.free_count, stream=stream)
