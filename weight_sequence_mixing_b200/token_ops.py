"""The operators beside the TTT layer (include/ttt_ops.h): rotary positions with several
axes, the gated linear recurrence, and group norm with an activation.

    rope = RotaryPositions(dict(d=64, pairs=(16, 16), base=100.0, dtype="bf16"))
    Q = rope.forward(q.view(B, N, H, d).transpose(1, 2), pos)   # heads first, for TTTLayer
    norm = GroupNorm(dict(C=H * d, groups=H, act="silu", dtype="bf16"))
    y = norm.forward(O, weight, bias)                           # O [B, H, N, d] -> [B, N, H d]
    scan = GatedScan(dict(D=H * d, gate="sigmoid", inp="complement", dtype="bf16"))
    h, state = scan.forward(gate, y, h0=state)

Every step runs in the CUDA library, on `stream` or else on the current stream of the object's
device; arguments are checked and marshalled by the module _token_ops, which raises ValueError
(TypeError for what is no tensor) before anything is enqueued, and TTTError with the library's
status.  Outputs that are not given are allocated on that stream, and so are workspaces, one for
each call: objects may be used on several streams and in several captured graphs at once.  The
calls do not synchronise and do not take part in autograd: `backward` is called with the gradients.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass, field

import torch

from .binding import DTYPE, LIB, TTT_ERR_CUDA, TTT_ERR_TIMEOUT, _check

try:
    from . import _token_ops as _native
except ImportError as e:
    raise ImportError("the module _token_ops is missing or does not fit this torch: build it with "
                      "weight_sequence_mixing_b200.build") from e

PAIRING = {"halves": 0, "interleaved": 1}
GATE = {"value": 0, "sigmoid": 1, "exp": 2}
SCAN_INPUT = {"plain": 0, "complement": 1}
ACT = {"none": 0, "silu": 1, "gelu": 2}
MAX_AXES = 4
_STATUS_TIMEOUT = 2


class RopeConfig(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("axes", ctypes.c_int32), ("pairs", ctypes.c_int32 * MAX_AXES),
                ("base", ctypes.c_double * MAX_AXES), ("pairing", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class ScanConfig(ctypes.Structure):
    _fields_ = [("D", ctypes.c_int32), ("gate", ctypes.c_int32), ("input", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class NormConfig(ctypes.Structure):
    _fields_ = [("C", ctypes.c_int32), ("groups", ctypes.c_int32), ("act", ctypes.c_int32), ("eps", ctypes.c_float),
                ("dtype", ctypes.c_int32)]


@dataclass
class _Op:
    """A configured operator: a C handle (host side only) bound to one device."""
    cfg: dict
    device: str = "cuda"
    _handle: ctypes.c_void_p = field(default=None, repr=False)

    _destroy = None
    _context = None  # of the handle, for _token_ops; None once closed

    def __post_init__(self):
        raise TypeError(f"{type(self).__name__} is not an operator of its own")

    def _open(self, create, destroy, config, a, b, status=False):
        dev = torch.device(self.device)
        if dev.type != "cuda":
            raise ValueError(f"device: expected a CUDA device, got {self.device}")
        self._index = dev.index
        if self._index is None:
            self._index = torch.cuda.current_device() if torch.cuda.is_available() else 0
        h = ctypes.c_void_p()
        _check(create(ctypes.byref(config), ctypes.byref(h)), create.__name__)
        self._handle, self._destroy = h, destroy
        if status:
            self._status = torch.zeros(1, dtype=torch.int32, device=f"cuda:{self._index}")
        self._context = _native.context(h.value, self._index, config.dtype == DTYPE["bf16"], a, b,
                                        self._status.data_ptr() if status else 0)

    def close(self):
        if self._handle:
            self._context = None
            self._destroy(self._handle)
            self._handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _on(self, stream, call, *args):
        """call(context, *args) on `stream`.  Tensors handed to another stream than the current one are
        kept from reuse until that stream is done with them."""
        if stream.device.index != self._index:
            raise ValueError(f"stream: expected one of cuda:{self._index}, got one of {stream.device}")
        for t in args:
            if isinstance(t, torch.Tensor) and t.is_cuda:
                t.record_stream(stream)
        with torch.cuda.stream(stream):
            return call(self._context, *args)


class _StatusOp(_Op):
    """An operator with a device status word, where a kernel that waits on other blocks reports a wait that ran out."""

    def check_status(self):
        """Waits for the device's work and raises if a call since the last check went wrong on the
        device (a bounded wait ran out; that call's outputs are not to be used)."""
        torch.cuda.synchronize(self._index)
        bits = int(self._status.item())
        if bits:
            self._status.zero_()
            _check(TTT_ERR_TIMEOUT if bits & _STATUS_TIMEOUT else TTT_ERR_CUDA, "device status")


class RotaryPositions(_Op):
    """Rotary positions with several axes.

    cfg: d (channels of a head), pairs (pairs of channels of each axis), base (one for all axes or one
    each; default 10000), pairing ("halves" or "interleaved"; default "halves"), dtype ("bf16", "f32").
    """

    def __post_init__(self):
        c, k = self.cfg, RopeConfig()
        pairs = list(c["pairs"])
        base = c.get("base", 10000.0)
        base = [float(v) for v in base] if isinstance(base, (list, tuple)) else [float(base)] * len(pairs)
        if not 1 <= len(pairs) <= MAX_AXES or len(base) != len(pairs):
            raise ValueError(f"pairs: expected 1 to {MAX_AXES} axes and a base for each, got {pairs} and {base}")
        k.d, k.axes = c["d"], len(pairs)
        for i, (n, b) in enumerate(zip(pairs, base)):
            k.pairs[i], k.base[i] = n, b
        k.pairing, k.dtype = PAIRING[c.get("pairing", "halves")], DTYPE[c["dtype"]]
        self._open(LIB.ttt_rope_create, LIB.ttt_rope_destroy, k, k.d, k.axes)

    def forward(self, x, pos, out=None, stream=None):
        """x [B, H, N, d] (any strides, channels contiguous) turned to its positions pos [N, axes] or
        [B, N, axes], int32 or float32.  out: given, and then possibly x itself, or a new contiguous tensor."""
        if stream is None:
            return _native.rope(self._context, x, pos, out, 0)
        return self._on(stream, _native.rope, x, pos, out, 0)

    def backward(self, dy, pos, out=None, stream=None):
        """The gradient of forward with respect to x: the rotation the other way."""
        if stream is None:
            return _native.rope(self._context, dy, pos, out, 1)
        return self._on(stream, _native.rope, dy, pos, out, 1)


class GatedScan(_StatusOp):
    """Gated linear recurrence h_t = a_t h_{t-1} + u_t over [B, L, D].

    cfg: D, gate ("value": a = g, "sigmoid": a = sigma(g), "exp": a = exp(g)), inp ("plain": u = x,
    "complement": u = (1 - a) x), dtype ("bf16", "f32").  States (h0, h_last and their gradients) are fp32 [B, D].
    """

    def __post_init__(self):
        c, k = self.cfg, ScanConfig()
        k.D, k.gate, k.input, k.dtype = c["D"], GATE[c["gate"]], SCAN_INPUT[c["inp"]], DTYPE[c["dtype"]]
        self._open(LIB.ttt_scan_create, LIB.ttt_scan_destroy, k, k.D, 0, status=True)

    def new_saved(self, B: int, L: int, stream=None):
        """A buffer for what a forward call leaves for its backward call."""
        if stream is None:
            return _native.scan_saved(self._context, B, L)
        return self._on(stream, _native.scan_saved, B, L)

    def forward(self, g, x, h0=None, lengths=None, saved=None, out=None, h_last=None, stream=None):
        """Returns (h [B, L, D], h_last [B, D]).  lengths: [B] int32, each sequence's own length; rows from
        there on are not used and are left as they were in `out` (zero where it is not given).  h_last may be h0."""
        if stream is None:
            return _native.scan_forward(self._context, g, x, h0, lengths, saved, out, h_last)
        return self._on(stream, _native.scan_forward, g, x, h0, lengths, saved, out, h_last)

    def backward(self, dh, g, x, saved, dh_last=None, lengths=None, dg=None, dx=None, dh0=None, stream=None):
        """Gradients (dg, dx [B, L, D], dh0 [B, D]) of a forward call with the same g, x and lengths that was
        given `saved`.  Rows behind a sequence's end are left as they were (zero in tensors made here)."""
        if stream is None:
            return _native.scan_backward(self._context, dh, g, x, saved, dh_last, lengths, dg, dx, dh0)
        return self._on(stream, _native.scan_backward, dh, g, x, saved, dh_last, lengths, dg, dx, dh0)


class GroupNorm(_StatusOp):
    """Group norm with an activation, channels last.

    cfg: C, groups, act ("none", "silu", "gelu"; default "none"), eps (default 1e-5), dtype ("bf16", "f32").
    x is [B, N, C], or [B, groups, N, C / groups] as TTTLayer returns it; y is [B, N, C].
    The statistics run over all N tokens of a call, later ones too: not for causal layers, nor for tokens that
    come one at a time.  Its kernels wait on no other block, so check_status finds nothing of theirs.
    """

    def __post_init__(self):
        c, k = self.cfg, NormConfig()
        k.C, k.groups, k.act, k.eps = c["C"], c["groups"], ACT[c.get("act", "none")], c.get("eps", 1e-5)
        k.dtype = DTYPE[c["dtype"]]
        self._open(LIB.ttt_norm_create, LIB.ttt_norm_destroy, k, k.C, k.groups, status=True)

    def new_stats(self, B: int, stream=None):
        """A buffer for the mean and 1 / sqrt(var + eps) of every group, for the backward call."""
        if stream is None:
            return _native.norm_stats(self._context, B)
        return self._on(stream, _native.norm_stats, B)

    def forward(self, x, weight=None, bias=None, stats=None, out=None, stream=None):
        """y [B, N, C].  weight, bias: [C] fp32.  out: given, and then possibly x itself, or new."""
        if stream is None:
            return _native.norm_forward(self._context, x, weight, bias, stats, out)
        return self._on(stream, _native.norm_forward, x, weight, bias, stats, out)

    def backward(self, dy, x, weight, bias, stats, dx=None, dweight=None, dbias=None, stream=None):
        """Gradients (dx of x's shape, dweight [C], dbias [C]) of a forward call that was given `stats`.
        dx: given, and then possibly dy itself, or new."""
        if stream is None:
            return _native.norm_backward(self._context, dy, x, weight, bias, stats, dx, dweight, dbias)
        return self._on(stream, _native.norm_backward, dy, x, weight, bias, stats, dx, dweight, dbias)
