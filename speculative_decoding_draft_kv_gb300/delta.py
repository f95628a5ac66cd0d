"""Thin Python binding of the C ABI declared in ``include/dflash_delta.h``: the gated delta rule
of recurrent layers, next to the paged-cache operators in :mod:`.paged`.

Two small handles describe what a serving program keeps anyway -- :class:`DeltaState` (a layer's
pool of states) and :class:`DeltaBatch` (the step's ragged batch) -- and each function has the
name of the C entry point that it calls.  Tensors are the caller's; the handles hold references to
theirs and nothing else.  Every call works on the current device and, unless given one, on its
current stream, and raises :class:`.ring.RingError` where the C call refuses.
"""

from __future__ import annotations

import ctypes

import torch

from .paged import _TYPES, _current_device, _device, _half, _packer, _rows, _stream, _vector, _workspace
from .ring import RING_EDEVICE, RING_OK, RingError, _load as _load_ring

DELTA_ERR_BATCH, DELTA_ERR_SLOT, DELTA_ERR_WAIT = 1, 2, 4

EXPORTED = ("delta_rule", "delta_rule_workspace", "delta_device_error", "delta_last_error")

_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class DeltaStateArgs(ctypes.Structure):
    _fields_ = ([("data", _vp)] + [(n, _i64) for n in ("slot_stride", "head_stride")] +
                [(n, _i32) for n in ("n_slots", "n_head", "dim_k", "dim_v")])


class DeltaBatchArgs(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("q_start", "slot_in", "slot_out", "save")] + [(n, _i32) for n in ("n_seq", "max_q")]


class DeltaRuleArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("state", "batch", "q", "k", "v", "o")] +
                [(n, _i64) for n in ("q_row_stride", "q_head_stride", "k_row_stride", "k_head_stride",
                                     "v_row_stride", "v_head_stride", "o_row_stride", "o_head_stride")] +
                [(n, _vp) for n in ("g", "beta")] + [(n, _i64) for n in ("g_row_stride", "beta_row_stride")] +
                [("workspace", _vp)] + [(n, _i64) for n in ("workspace_bytes", "n_rows")] +
                [(n, _f32) for n in ("scale", "eps")] + [(n, _i32) for n in ("n_head_k", "dtype", "normalise", "reserved")])


_pack_rule = _packer(DeltaRuleArgs)
_LIB = None


def _load():
    global _LIB
    if _LIB is None:
        lib = _load_ring()
        lib.delta_rule.argtypes = [_vp, _vp]
        lib.delta_rule_workspace.argtypes = [_vp, _vp, _i64, _i32, ctypes.POINTER(_i64)]
        lib.delta_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint32)]
        lib.delta_last_error.restype = ctypes.c_char_p
        _LIB = lib
    return _LIB


def delta_last_error() -> str:
    return _load().delta_last_error().decode()


def _check(rc):
    if rc != RING_OK:
        raise RingError(rc, delta_last_error())


class DeltaState:
    """A layer's pool of states: float32 [n_slots, n_head, dim_v, dim_k] (any slot and head strides, rows contiguous)."""

    def __init__(self, state):
        self.device = _device(state, "state")
        if state.dim() != 4 or state.dtype != torch.float32:
            raise TypeError("state must be float32 [n_slots, n_head, dim_v, dim_k]")
        n_slots, self.n_head, self.dim_v, self.dim_k = state.shape
        if state.numel() and (state.stride(3) != 1 or state.stride(2) != self.dim_k):
            raise ValueError("a head's rows must be contiguous")
        # strides of dimensions of one entry say nothing
        size = self.dim_v * self.dim_k
        head = state.stride(1) if self.n_head > 1 else size
        slot = state.stride(0) if n_slots > 1 else max(head, size) * max(1, self.n_head)
        self.tensors = (state,)
        self.args = DeltaStateArgs(state.data_ptr(), slot, head, n_slots, self.n_head, self.dim_k, self.dim_v)
        self.address = ctypes.addressof(self.args)


class DeltaBatch:
    """A ragged batch of new tokens (the C struct ``delta_batch``).  ``q_start``: int32
    [n_seq + 1], ``slot_in``, ``slot_out``: int32 [n_seq], ``save``: None or int32 [rows], on the
    device; ``max_q``: host bound of a sequence's new tokens now and at every replay of a captured
    call.  A batch with ``save`` goes token by token, whatever its lengths: prompts want a batch of their own."""

    def __init__(self, q_start, slot_in, slot_out, max_q, save=None):
        self.device = _device(q_start, "q_start")
        n = slot_in.shape[0]
        _vector(q_start, "q_start", torch.int32, n + 1, self.device)
        _vector(slot_in, "slot_in", torch.int32, n, self.device)
        _vector(slot_out, "slot_out", torch.int32, n, self.device)
        if save is not None:
            _vector(save, "save", torch.int32, save.numel(), self.device)
        if not 0 <= max_q < 1 << 30:
            raise ValueError(f"max_q {max_q} out of range")
        self.rows = None if save is None else save.numel()
        self.tensors = (q_start, slot_in, slot_out, save)
        self.args = DeltaBatchArgs(q_start.data_ptr(), slot_in.data_ptr(), slot_out.data_ptr(),
                                   None if save is None else save.data_ptr(), n, int(max_q))
        self.address = ctypes.addressof(self.args)


def _one_device(state, batch):
    d = _current_device()
    if state.device != d or batch.device != d:
        raise ValueError(f"state (device {state.device}) and batch (device {batch.device}) must be on the current "
                         f"device, {d}")
    return d


def _scalars(t, name, n, heads, device):
    """(pointer, row stride) of a float32 tensor [n, heads] with contiguous heads."""
    if t.dtype is not torch.float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    if t.shape != (n, heads) or t.get_device() != device or (heads > 1 and n and t.stride(1) != 1):
        raise ValueError(f"{name} must be [{n}, {heads}] with contiguous heads on device {device}")
    return t.data_ptr(), t.stride(0) if n > 1 else 0


def delta_rule_workspace(state, batch, n_rows, n_head_k) -> int:
    """Bytes of workspace that :func:`delta_rule` needs."""
    _one_device(state, batch)
    n = _i64()
    _check(_load().delta_rule_workspace(state.address, batch.address, int(n_rows), int(n_head_k), ctypes.byref(n)))
    return n.value


def delta_rule(state, batch, q, k, v, g, beta, o, normalise=True, eps=1e-6, scale=0.0, workspace=None, stream=None):
    """``q``, ``k``: float16 or bfloat16 [rows, n_head_k, dim_k]; ``v``, ``o``: the same type
    [rows, n_head, dim_v]; ``g`` (log decays), ``beta``: float32 [rows, n_head]; ``normalise``: q
    and k are divided by sqrt(sum of squares + ``eps``) first; ``scale``: of q, 0 for
    1 / sqrt(dim_k).  ``workspace``: a uint8 tensor of :func:`delta_rule_workspace` bytes that no
    other call uses at the same time, or None for one of the call's own from PyTorch's allocator."""
    dev = _one_device(state, batch)
    n, heads_k, dtype = q.shape[0], q.shape[1], q.dtype
    qp, qr, qh = _rows(q, "q", n, heads_k, state.dim_k, _half(dtype), dev)
    kp, kr, kh = _rows(k, "k", n, heads_k, state.dim_k, dtype, dev)
    vp, vr, vh = _rows(v, "v", n, state.n_head, state.dim_v, dtype, dev)
    op, orow, oh = _rows(o, "o", n, state.n_head, state.dim_v, dtype, dev)
    gp, gr = _scalars(g, "g", n, state.n_head, dev)
    bp, br = _scalars(beta, "beta", n, state.n_head, dev)
    if batch.rows is not None and batch.rows != n:
        raise ValueError(f"save must have {n} entries, got {batch.rows}")
    st = _stream(stream, dev)
    workspace = _workspace(workspace, lambda: delta_rule_workspace(state, batch, n, heads_k), st, stream, dev, q.device)
    a = _pack_rule(state.address, batch.address, qp, kp, vp, op, qr, qh, kr, kh, vr, vh, orow, oh, gp, bp, gr, br,
                   workspace.data_ptr(), workspace.numel(), n, scale, eps, heads_k, _TYPES[dtype], bool(normalise), 0)
    _check(_load().delta_rule(a, st))


def delta_device_error() -> int:
    """Synchronise, read and clear the operator's error word (DELTA_ERR_* bits; 0: none)."""
    bits = ctypes.c_uint32()
    rc = _load().delta_device_error(ctypes.byref(bits))
    if rc not in (RING_OK, RING_EDEVICE):
        _check(rc)
    return bits.value
