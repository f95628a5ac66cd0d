"""Thin Python binding of the C ABI declared in ``include/dflash_paged.h``: operators over a
paged K/V cache, next to the ring's in :mod:`.ring`.

Three small handles describe what a serving program keeps anyway -- :class:`PagedCache` (one
layer's pools), :class:`PagedBatch` (the step's ragged batch) and :class:`PagedRope` (the
rotation's frequencies) -- and each function has the name of the C entry point that it calls.
Tensors are the caller's; the handles hold references to theirs and nothing else.  Every call
works on the current device and, unless given one, on its current stream, and raises
:class:`.ring.RingError` where the C call refuses.
"""

from __future__ import annotations

import ctypes
import math
import struct

import torch

from .ring import RING_EDEVICE, RING_OK, RingError, _load as _load_ring

PAGED_F16, PAGED_BF16, PAGED_F32, PAGED_INT8, PAGED_E4M3 = range(5)
PAGED_CAUSAL, PAGED_FULL, PAGED_TREE = range(3)
PAGED_HALF, PAGED_INTERLEAVED = range(2)
PAGED_ERR_WAIT, PAGED_ERR_PAGE = 1, 2
MASKS = {"causal": PAGED_CAUSAL, "full": PAGED_FULL, "tree": PAGED_TREE}
LAYOUTS = {"half": PAGED_HALF, "interleaved": PAGED_INTERLEAVED}
_TYPES = {torch.float16: PAGED_F16, torch.bfloat16: PAGED_BF16, torch.float32: PAGED_F32,
          torch.int8: PAGED_INT8, torch.float8_e4m3fn: PAGED_E4M3}

EXPORTED = ("paged_rope_init", "paged_norm_rope", "paged_append", "paged_gather", "paged_attend", "paged_attend_workspace",
            "paged_attend_shared", "paged_attend_shared_workspace", "paged_device_error", "paged_last_error")

_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class PagedCacheArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("k", "v", "k_scale", "v_scale")] +
                [(n, _i64) for n in ("page_stride", "head_stride", "row_stride", "scale_page_stride",
                                     "scale_head_stride")] +
                [(n, _i32) for n in ("n_pages", "page_size", "n_head_kv", "head_dim", "format", "reserved")])


class PagedBatchArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("q_start", "kv_len", "pages")] + [("pages_stride", _i64)] +
                [(n, _i32) for n in ("n_seq", "max_pages", "max_q", "max_kv")])


class PagedRopeArgs(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_uint64 * 64), ("magnitude", _f32), ("rotary_dim", _i32), ("layout", _i32),
                ("reserved", _i32)]


class PagedNormRopeArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("q", "k", "q_out", "k_out")] +
                [(n, _i64) for n in ("q_row_stride", "q_head_stride", "k_row_stride", "k_head_stride",
                                     "qo_row_stride", "qo_head_stride", "ko_row_stride", "ko_head_stride")] +
                [(n, _vp) for n in ("q_norm", "k_norm", "positions", "rope")] + [("n_rows", _i64), ("eps", _f32)] +
                [(n, _i32) for n in ("n_head_q", "n_head_k", "head_dim", "dtype")])


class PagedAppendArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("cache", "batch", "k", "v", "q", "q_out")] +
                [(n, _i64) for n in ("k_row_stride", "k_head_stride", "v_row_stride", "v_head_stride",
                                     "q_row_stride", "q_head_stride", "qo_row_stride", "qo_head_stride")] +
                [(n, _vp) for n in ("k_norm", "q_norm", "positions", "rope")] + [("n_rows", _i64), ("eps", _f32)] +
                [(n, _i32) for n in ("n_head_q", "dtype")])


class PagedGatherArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("cache", "batch", "k", "v")] +
                [(n, _i64) for n in ("k_row_stride", "k_head_stride", "v_row_stride", "v_head_stride", "n_rows")] +
                [(n, _i32) for n in ("dtype", "reserved")])


class PagedAttendArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("cache", "batch", "q", "o")] +
                [(n, _i64) for n in ("q_row_stride", "q_head_stride", "o_row_stride", "o_head_stride")] +
                [(n, _vp) for n in ("tree", "lse", "workspace")] + [(n, _i64) for n in ("workspace_bytes", "n_rows")] +
                [("scale", _f32)] + [(n, _i32) for n in ("n_head", "dtype", "mask", "window", "reserved")])



def _packer(args):
    """The struct's fields to its bytes, as an address argument takes them (a tenth of a call's time less than
    making the ctypes object)."""
    codes = {_vp: "Q", _i64: "q", _i32: "i", _f32: "f"}
    s = struct.Struct("@" + "".join(codes[t] for _, t in args._fields_))
    assert s.size == ctypes.sizeof(args)

    def pack(*values):
        try:
            return s.pack(*values)
        except struct.error as e:
            raise TypeError(f"{args.__name__}: {e}") from None
    return pack


_pack_attend = _packer(PagedAttendArgs)
_LIB = None


def _load():
    global _LIB
    if _LIB is None:
        lib = _load_ring()
        for name in ("paged_norm_rope", "paged_append", "paged_gather", "paged_attend"):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = [_vp, _vp], ctypes.c_int
        lib.paged_rope_init.argtypes = [_vp, ctypes.POINTER(ctypes.c_double), ctypes.c_double, _i32, _i32]
        lib.paged_attend_workspace.argtypes = [_vp, _vp, _i32, ctypes.POINTER(_i64)]
        lib.paged_attend_shared.argtypes = [_vp, _vp, _vp]
        lib.paged_attend_shared_workspace.argtypes = [_vp, _vp, _vp, _i64, _i32, ctypes.POINTER(_i64)]
        lib.paged_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint32)]
        lib.paged_last_error.restype = ctypes.c_char_p
        _LIB = lib
    return _LIB


def paged_last_error() -> str:
    return _load().paged_last_error().decode()


def _check(rc):
    if rc != RING_OK:
        raise RingError(rc, paged_last_error())


def _device(t, name):
    """The tensor's device index, refused where it is not the current device."""
    d = t.get_device()
    if d < 0:
        raise TypeError(f"{name} must be a CUDA tensor")
    if d != torch.cuda.current_device():
        raise ValueError(f"{name} is on device {d}, the current device is {torch.cuda.current_device()}")
    return d


# The current device, and the handle of PyTorch's current stream without the Python object around it (1 us of a call of 8).
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda device: torch.cuda.current_stream(device).cuda_stream)


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream, device):
    if stream is None:
        return _current_stream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _rows(t, name, n, heads, dim, dtype, device):
    """(pointer, row stride, head stride) of a rows tensor [n, heads, dim]."""
    s = t.stride()
    if t.shape != (n, heads, dim) or t.dtype is not dtype or t.get_device() != device or s[2] != 1:
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        raise ValueError(f"{name} must be [{n}, {heads}, {dim}] with contiguous heads on device {device}, got "
                         f"{tuple(t.shape)} with strides {s} on device {t.get_device()}")
    # strides of dimensions of one entry say nothing
    return t.data_ptr(), s[0] if n > 1 else 0, s[1] if heads > 1 else 0


def _vector(t, name, dtype, n, device):
    """Pointer of a contiguous tensor of n entries."""
    if t.dtype is not dtype or t.numel() != n or t.get_device() != device or not t.is_contiguous():
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        raise ValueError(f"{name} must be contiguous with {n} entries on device {device}")
    return t.data_ptr()


class PagedCache:
    """One layer's pools.  ``k``, ``v``: [n_pages, n_head_kv, page_size, head_dim] (any strides
    with contiguous heads; a [n_pages, page_size, n_head_kv, head_dim] pool is given as its
    transpose(1, 2)) of float16, bfloat16, int8 or float8_e4m3fn; for the last two ``k_scale``,
    ``v_scale``: float32 [n_pages, n_head_kv, page_size]."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        self.device = _device(k, "k")
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or v.get_device() != self.device:
            raise ValueError("k and v must be [n_pages, n_head_kv, page_size, head_dim] alike")
        if k.dtype not in _TYPES or k.dtype == torch.float32:
            raise TypeError(f"unknown page type {k.dtype}")
        if k.stride() != v.stride() or k.stride(3) != 1:
            raise ValueError("k and v must have the same strides and contiguous heads")
        self.format, self.dtype = _TYPES[k.dtype], k.dtype
        self.coded = self.format in (PAGED_INT8, PAGED_E4M3)
        n_pages, self.n_head_kv, page_size, self.head_dim = k.shape
        sp = sh = 0
        if self.coded:
            for t in (k_scale, v_scale):
                if t is None or t.dtype != torch.float32 or t.shape != k.shape[:3] or t.get_device() != self.device:
                    raise ValueError("quantised pages need float32 scales [n_pages, n_head_kv, page_size]")
                if t.stride(2) != 1 or t.stride() != k_scale.stride():
                    raise ValueError("scales must be contiguous within a page, k's and v's alike")
            sp, sh = k_scale.stride(0), k_scale.stride(1)
        elif k_scale is not None or v_scale is not None:
            raise ValueError("16-bit pages have no scales")
        self.tensors = (k, v, k_scale, v_scale)
        self.args = PagedCacheArgs(k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if self.coded else None,
                                   v_scale.data_ptr() if self.coded else None, k.stride(0), k.stride(1), k.stride(2),
                                   sp, sh, n_pages, page_size, self.n_head_kv, self.head_dim, self.format, 0)
        self.address = ctypes.addressof(self.args)


class PagedBatch:
    """A ragged batch of new tokens (the C struct ``paged_batch``).  ``q_start``: int32
    [n_seq + 1], ``kv_len``: int32 [n_seq], ``pages``: int32 [n_seq, max_pages], on the device;
    ``max_q``, ``max_kv``: host bounds of what they hold now and at every replay of a captured
    call (``max_kv`` default: all that the block table spans)."""

    def __init__(self, q_start, kv_len, pages, max_q, max_kv=0):
        self.device = _device(q_start, "q_start")
        n = kv_len.shape[0]
        _vector(q_start, "q_start", torch.int32, n + 1, self.device)
        _vector(kv_len, "kv_len", torch.int32, n, self.device)
        if pages.dim() != 2 or pages.shape[0] != n or pages.dtype != torch.int32 or pages.get_device() != self.device:
            raise ValueError(f"pages must be int32 [{n}, max_pages] on the batch's device")
        if pages.shape[1] > 1 and pages.stride(1) != 1:
            raise ValueError("a row of pages must be contiguous")
        if not (0 <= max_q < 1 << 30 and 0 <= max_kv < 1 << 30):
            raise ValueError(f"max_q {max_q} or max_kv {max_kv} out of range")
        self.tensors = (q_start, kv_len, pages)
        self.args = PagedBatchArgs(q_start.data_ptr(), kv_len.data_ptr(), pages.data_ptr(), pages.stride(0), n,
                                   pages.shape[1], int(max_q), int(max_kv))
        self.address = ctypes.addressof(self.args)


def rope_frequencies(rotary_dim, theta, scaling="none", factor=1.0, original_len=0, beta_fast=32.0, beta_slow=1.0):
    """(angle per position of each pair, magnitude) of a rotation.

    ``scaling``: "none"; "linear" (positions divided by ``factor``); "ntk" (theta multiplied by
    factor^(r / (r - 2)), which slows the lowest frequency by ``factor`` and leaves the highest);
    "yarn" (by parts: pairs that turn more than ``beta_fast`` times within ``original_len``
    positions stay, those that turn less than ``beta_slow`` times slow down by ``factor``, a ramp
    linear in the number of turns between; magnitude 0.1 ln(factor) + 1).  Programs that make the ramp
    linear in the pair's index instead, between borders that they may round, give other
    frequencies to the pairs between: weights that were trained or run so want those, as
    :class:`PagedRope`'s ``inv_freq`` and ``magnitude``.
    """
    r = int(rotary_dim)
    if r <= 0 or r % 2 or not theta > 0 or not factor > 0:
        raise ValueError("rotary_dim must be even and positive, theta and factor positive")
    if scaling == "ntk":
        if r < 4:
            raise ValueError("ntk scaling needs rotary_dim of at least 4")
        theta = theta * factor ** (r / (r - 2))
    freq = [theta ** (-2.0 * i / r) for i in range(r // 2)]
    if scaling in ("none", "ntk"):
        return freq, 1.0
    if scaling == "linear":
        return [f / factor for f in freq], 1.0
    if scaling == "yarn":
        if original_len <= 0 or not beta_fast > beta_slow:
            raise ValueError("yarn scaling needs original_len, and beta_fast above beta_slow")
        keep = [min(1.0, max(0.0, (original_len * f / (2 * math.pi) - beta_slow) / (beta_fast - beta_slow)))
                for f in freq]
        return [(1 - g) * f / factor + g * f for g, f in zip(keep, freq)], 0.1 * math.log(factor) + 1.0
    raise ValueError(f"unknown scaling {scaling!r}")


class PagedRope:
    """A position rotation: the first ``rotary_dim`` elements of a head in "half" (i, i + r/2) or
    "interleaved" (2i, 2i + 1) pairs, with :func:`rope_frequencies`' frequencies or the caller's
    ``inv_freq`` and ``magnitude``."""

    def __init__(self, rotary_dim, theta=1.0e4, layout="half", scaling="none", factor=1.0, original_len=0,
                 beta_fast=32.0, beta_slow=1.0, inv_freq=None, magnitude=1.0):
        if inv_freq is None:
            inv_freq, magnitude = rope_frequencies(rotary_dim, theta, scaling, factor, original_len, beta_fast,
                                                   beta_slow)
        if len(inv_freq) != rotary_dim // 2:
            raise ValueError(f"inv_freq must have {rotary_dim // 2} entries, got {len(inv_freq)}")
        self.inv_freq, self.magnitude = [float(f) for f in inv_freq], float(magnitude)
        self.args = PagedRopeArgs()
        _check(_load().paged_rope_init(self.address, (ctypes.c_double * len(self.inv_freq))(*self.inv_freq),
                                       self.magnitude, rotary_dim, LAYOUTS.get(layout, layout)))

    @property
    def address(self):
        """Of the struct that this handle holds: a copy (of a model's, or sent to another process) has its own."""
        return ctypes.addressof(self.args)


_ROW_TYPES = (torch.float16, torch.bfloat16, torch.float32)


def _one_device(cache, batch):
    d = _current_device()
    if cache.device != d or batch.device != d:
        raise ValueError(f"cache (device {cache.device}) and batch (device {batch.device}) must be on the current "
                         f"device, {d}")
    return d


def _half(dtype):
    if dtype is not torch.float16 and dtype is not torch.bfloat16:
        raise TypeError(f"rows must be float16 or bfloat16, got {dtype}")
    return dtype


def paged_norm_rope(positions, rope, eps=1e-6, q=None, q_norm=None, q_out=None, k=None, k_norm=None, k_out=None,
                    stream=None):
    """``q``, ``k``: float16, bfloat16 or float32 [rows, heads, head_dim], either may be left out;
    ``*_out``: the same shape and type (or the tensor itself); ``*_norm``: float32 [head_dim] or
    None; ``positions``: int32 [rows]; ``rope``: a :class:`PagedRope` or None."""
    lead = q if q is not None else k
    if lead is None or (q is None) != (q_out is None) or (k is None) != (k_out is None):
        raise ValueError("give q, k or both, each with its output")
    dev = _device(lead, "q" if q is not None else "k")
    dtype, shape = lead.dtype, lead.shape
    if len(shape) != 3 or dtype not in _ROW_TYPES:
        raise TypeError("q and k must be float16, bfloat16 or float32 [rows, heads, head_dim]")
    n, _, dim = shape
    q_ptr = qo_ptr = k_ptr = ko_ptr = qn = kn = None
    q_row = q_head = qo_row = qo_head = k_row = k_head = ko_row = ko_head = nq = nk = 0
    if q is not None:
        nq = q.shape[1]
        q_ptr, q_row, q_head = _rows(q, "q", n, nq, dim, dtype, dev)
        qo_ptr, qo_row, qo_head = _rows(q_out, "q_out", n, nq, dim, dtype, dev)
        if q_norm is not None:
            qn = _vector(q_norm, "q_norm", torch.float32, dim, dev)
    if k is not None:
        nk = k.shape[1]
        k_ptr, k_row, k_head = _rows(k, "k", n, nk, dim, dtype, dev)
        ko_ptr, ko_row, ko_head = _rows(k_out, "k_out", n, nk, dim, dtype, dev)
        if k_norm is not None:
            kn = _vector(k_norm, "k_norm", torch.float32, dim, dev)
    a = PagedNormRopeArgs(q_ptr, k_ptr, qo_ptr, ko_ptr, q_row, q_head, k_row, k_head, qo_row, qo_head, ko_row, ko_head,
                          qn, kn, None if positions is None else _vector(positions, "positions", torch.int32, n, dev),
                          None if rope is None else rope.address, n, eps, nq, nk, dim, _TYPES[dtype])
    _check(_load().paged_norm_rope(ctypes.addressof(a), _stream(stream, dev)))


def paged_append(cache, batch, k, v, rope=None, eps=1e-6, k_norm=None, q=None, q_norm=None, q_out=None,
                 positions=None, stream=None):
    """Write the batch's ``k``, ``v`` rows (float16 or bfloat16 [rows, n_head_kv, head_dim]) into
    the cache's pages, K normed and turned first where ``k_norm`` and ``rope`` say so, at its
    position in the sequence or at ``positions`` (int32 [rows]); with ``q`` and ``q_out`` the
    queries are normed (``q_norm``) and turned in the same pass."""
    dev = _one_device(cache, batch)
    dim, heads, n, dtype = cache.head_dim, cache.n_head_kv, k.shape[0], k.dtype
    if (q is None) != (q_out is None):
        raise ValueError("q goes with q_out")
    k_ptr, k_row, k_head = _rows(k, "k", n, heads, dim, _half(dtype), dev)
    v_ptr, v_row, v_head = _rows(v, "v", n, heads, dim, dtype, dev)
    q_ptr = qo_ptr = qn = None
    q_row = q_head = qo_row = qo_head = nq = 0
    if q is not None:
        nq = q.shape[1]
        q_ptr, q_row, q_head = _rows(q, "q", n, nq, dim, dtype, dev)
        qo_ptr, qo_row, qo_head = _rows(q_out, "q_out", n, nq, dim, dtype, dev)
        if q_norm is not None:
            qn = _vector(q_norm, "q_norm", torch.float32, dim, dev)
    a = PagedAppendArgs(cache.address, batch.address, k_ptr, v_ptr, q_ptr, qo_ptr, k_row, k_head, v_row, v_head, q_row,
                        q_head, qo_row, qo_head, None if k_norm is None else _vector(k_norm, "k_norm", torch.float32, dim, dev),
                        qn, None if positions is None else _vector(positions, "positions", torch.int32, n, dev),
                        None if rope is None else rope.address, n, eps, nq, _TYPES[dtype])
    _check(_load().paged_append(ctypes.addressof(a), _stream(stream, dev)))


def paged_gather(cache, batch, k, v, stream=None):
    """Read the batch's rows back into ``k``, ``v`` (float16 or bfloat16 [rows, n_head_kv, head_dim])."""
    dev = _one_device(cache, batch)
    dim, heads, n, dtype = cache.head_dim, cache.n_head_kv, k.shape[0], k.dtype
    kp, kr, kh = _rows(k, "k", n, heads, dim, _half(dtype), dev)
    vp, vr, vh = _rows(v, "v", n, heads, dim, dtype, dev)
    a = PagedGatherArgs(cache.address, batch.address, kp, vp, kr, kh, vr, vh, n, _TYPES[dtype], 0)
    _check(_load().paged_gather(ctypes.addressof(a), _stream(stream, dev)))


def _workspace(given, size, st, stream, dev, device):
    """The workspace given, or one of size() bytes for stream ``st``."""
    if given is None:
        # from the pool of the stream that the work runs on, which alone may have it next
        if stream is None:
            return torch.empty(size(), dtype=torch.uint8, device=device)
        with torch.cuda.stream(torch.cuda.ExternalStream(st) if st else torch.cuda.default_stream(dev)):
            return torch.empty(size(), dtype=torch.uint8, device=device)
    if given.get_device() != dev or given.dtype != torch.uint8 or not given.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 CUDA tensor of the call's device")
    return given


def paged_attend_workspace(cache, batch, n_head) -> int:
    """Bytes of workspace that :func:`paged_attend` needs."""
    _one_device(cache, batch)
    n = _i64()
    _check(_load().paged_attend_workspace(cache.address, batch.address, int(n_head), ctypes.byref(n)))
    return n.value


def paged_attend(cache, batch, q, o, mask="causal", window=0, scale=0.0, tree=None, lse=None, workspace=None,
                 stream=None):
    """``q``, ``o``: float16 or bfloat16 [rows, n_head, head_dim]; ``mask``: "causal", "full" or
    "tree" (with ``tree``: int64 [rows], bit j of a token's word: it sees the sequence's j-th new
    token); ``window``: 0 or the length of a sliding window; ``lse``: None or float32
    [rows, n_head].  ``workspace``: a uint8 tensor of :func:`paged_attend_workspace` bytes that no
    other call uses at the same time, or None for one of the call's own from PyTorch's allocator."""
    a, st, workspace = _attend_args(cache, batch, q, o, mask, window, scale, tree, lse, workspace, stream,
                                    lambda n, heads: paged_attend_workspace(cache, batch, heads))
    _check(_load().paged_attend(a, st))


def _attend_args(cache, batch, q, o, mask, window, scale, tree, lse, workspace, stream, size):
    """(the call's struct as bytes, stream, workspace, to be kept until the call is made); size(rows, heads): its bytes."""
    dev = _one_device(cache, batch)
    dtype, (n, heads, _) = q.dtype, q.shape
    qp, qr, qh = _rows(q, "q", n, heads, cache.head_dim, _half(dtype), dev)
    op, orow, oh = _rows(o, "o", n, heads, cache.head_dim, dtype, dev)
    tp = 0 if tree is None else _vector(tree, "tree", torch.int64, n, dev)
    lp = 0 if lse is None else _vector(lse, "lse", torch.float32, n * heads, dev)
    if not 0 <= window < 1 << 31:
        raise ValueError(f"window {window} out of range")
    st = _stream(stream, dev)
    workspace = _workspace(workspace, lambda: size(n, heads), st, stream, dev, q.device)
    return _pack_attend(cache.address, batch.address, qp, op, qr, qh, orow, oh, tp, lp, workspace.data_ptr(), workspace.numel(),
                        n, scale, heads, _TYPES[dtype], MASKS.get(mask, mask), window, 0), st, workspace


def paged_attend_shared_workspace(cache, batch, prefix, n_rows, n_head) -> int:
    """Bytes of workspace that :func:`paged_attend_shared` needs."""
    _one_device(cache, batch)
    _one_device(cache, prefix)
    n = _i64()
    _check(_load().paged_attend_shared_workspace(cache.address, batch.address, prefix.address, int(n_rows), int(n_head),
                                                 ctypes.byref(n)))
    return n.value


def paged_attend_shared(cache, batch, prefix, q, o, mask="causal", scale=0.0, tree=None, lse=None, workspace=None,
                        stream=None):
    """:func:`paged_attend` for sequences that share beginnings: ``batch`` describes what each has of its own (``kv_len``
    and ``pages`` count from behind the beginning), ``prefix`` -- a :class:`PagedBatch` too -- the beginnings:
    ``q_start``: bounds of the rows that have each one, ``kv_len``: their lengths, ``pages``: where they lie; ``max_q``:
    bound of one's rows."""
    _one_device(cache, prefix)
    a, st, workspace = _attend_args(cache, batch, q, o, mask, 0, scale, tree, lse, workspace, stream,
                                    lambda n, heads: paged_attend_shared_workspace(cache, batch, prefix, n, heads))
    _check(_load().paged_attend_shared(a, prefix.address, st))


def paged_device_error() -> int:
    """Synchronise, read and clear the operators' error word (PAGED_ERR_* bits; 0: none)."""
    bits = ctypes.c_uint32()
    rc = _load().paged_device_error(ctypes.byref(bits))
    if rc not in (RING_OK, RING_EDEVICE):
        _check(rc)
    return bits.value
