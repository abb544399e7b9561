"""The operators beside the TTT layer (include/ttt_ops.h): rotary positions with several
axes, the gated linear recurrence, and group norm with an activation.

    rope = RotaryPositions(dict(d=64, pairs=(16, 16), base=100.0, dtype="bf16"))
    Q = rope.forward(q.view(B, N, H, d).transpose(1, 2), pos)   # heads first, for TTTLayer
    norm = GroupNorm(dict(C=H * d, groups=H, act="silu", dtype="bf16"))
    y = norm.forward(O, weight, bias)                           # O [B, H, N, d] -> [B, N, H d]
    scan = GatedScan(dict(D=H * d, gate="sigmoid", inp="complement", dtype="bf16"))
    h, state = scan.forward(gate, y, h0=state)

As with TTTLayer, arguments are checked and marshalled here and every step runs in the CUDA
library, on `stream` or else on the current stream of the object's device.  Outputs that are
not given are allocated on that stream, and so are workspaces, one for each call: objects
may be used on several streams and in several captured graphs at once.  The calls do not
synchronise and do not take part in autograd: `backward` is called with the gradients.
"""
from __future__ import annotations

import ctypes
from contextlib import nullcontext
from dataclasses import dataclass, field

import torch

from .binding import DTYPE, LIB, TTT_ERR_TIMEOUT, _check

PAIRING = {"halves": 0, "interleaved": 1}
GATE = {"value": 0, "sigmoid": 1, "exp": 2}
SCAN_INPUT = {"plain": 0, "complement": 1}
ACT = {"none": 0, "silu": 1, "gelu": 2}
POS_DTYPE = {torch.int32: 0, torch.float32: 1}
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


_STRIDES: dict = {}


def _strides(batch: int, head: int, token: int):
    """A ttt_strides of these values (kept: a program has few, and a call needs several)."""
    key = (batch, head, token)
    s = _STRIDES.get(key)
    if s is None:
        if len(_STRIDES) >= 4096:
            _STRIDES.clear()
        s = _STRIDES[key] = (ctypes.c_int64 * 3)(batch, head, token)
    return s


def _ptr(t):
    return None if t is None else t.data_ptr()


@dataclass
class _Op:
    """A configured operator: a C handle (host side only) bound to one device."""
    cfg: dict
    device: str = "cuda"
    _handle: ctypes.c_void_p = field(default=None, repr=False)

    _destroy = None

    def __post_init__(self):
        raise TypeError(f"{type(self).__name__} is not an operator of its own")

    def _open(self, create, destroy, config):
        h = ctypes.c_void_p()
        _check(create(ctypes.byref(config), ctypes.byref(h)), create.__name__)
        self._handle = h
        self._destroy = destroy
        self.io_dtype = torch.float32 if self.cfg["dtype"] == "f32" else torch.bfloat16
        dev = torch.device(self.device)
        if dev.type != "cuda":
            raise ValueError(f"device: expected a CUDA device, got {self.device}")
        self._index = dev.index if dev.index is not None or not torch.cuda.is_available() else \
            torch.cuda.current_device()

    def close(self):
        if self._handle:
            self._destroy(self._handle)
            self._handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _need_open(self):
        if not self._handle:
            raise ValueError(f"{type(self).__name__} is closed")

    def _tensor(self, name, t, shape, dtype, rows=True):
        """`t` is on this device, with this shape and dtype; its rows (rows=True) or all of it contiguous."""
        if t.dtype != dtype or t.shape != shape:
            raise ValueError(f"{name}: expected shape {tuple(shape)} of {dtype}, got {tuple(t.shape)} of {t.dtype}")
        if not t.is_cuda or t.device.index != self._index:
            raise ValueError(f"{name}: expected a tensor on cuda:{self._index}, got one on {t.device}")
        if rows:
            if t.stride(-1) != 1 and t.shape[-1] > 1:
                raise ValueError(f"{name}: the channels of a row must be contiguous, got strides {t.stride()}")
        elif not t.is_contiguous():
            raise ValueError(f"{name}: must be contiguous")

    def _on(self, stream, *tensors):
        """The context to allocate and launch in.  Tensors handed to another stream than the
        current one are kept from reuse until that stream is done with them."""
        if stream is None:
            return nullcontext() if torch.cuda.current_device() == self._index else torch.cuda.device(self._index)
        if stream.device.index != self._index:
            raise ValueError(f"stream: expected one of cuda:{self._index}, got one of {stream.device}")
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
        return torch.cuda.stream(stream)

    def _stream(self):
        return torch.cuda.current_stream(self._index).cuda_stream


class _StatusOp(_Op):
    """An operator whose kernels wait on one another and report a wait that ran out."""

    def _open(self, create, destroy, config):
        super()._open(create, destroy, config)
        self._status = torch.zeros(1, dtype=torch.int32, device=f"cuda:{self._index}")

    def check_status(self):
        """Waits for the device's work and raises if a call since the last check went wrong on the
        device (a bounded wait ran out; the call's outputs hold NaN where they are unknown)."""
        torch.cuda.synchronize(self._index)
        bits = int(self._status.item())
        if bits:
            self._status.zero_()
            _check(TTT_ERR_TIMEOUT if bits & _STATUS_TIMEOUT else -3, "device status")


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
        self.axes = len(pairs)
        self._open(LIB.ttt_rope_create, LIB.ttt_rope_destroy, k)

    def _apply(self, x, pos, out, inverse, stream, name):
        self._need_open()
        if x.dim() != 4:
            raise ValueError(f"{name}: expected [B, H, N, {self.cfg['d']}], got shape {tuple(x.shape)}")
        B, H, N, _ = shape = x.shape
        self._tensor(name, x, (B, H, N, self.cfg["d"]), self.io_dtype)
        if pos.dtype not in POS_DTYPE or pos.shape not in ((N, self.axes), (B, N, self.axes)):
            raise ValueError(f"pos: expected [{N}, {self.axes}] or [{B}, {N}, {self.axes}] of int32 or float32, got "
                             f"shape {tuple(pos.shape)} of {pos.dtype}")
        self._tensor("pos", pos, pos.shape, pos.dtype, rows=False)
        with self._on(stream, x, pos, out):
            if out is None:
                out = torch.empty(shape, dtype=self.io_dtype, device=x.device)
            else:
                self._tensor("out", out, shape, self.io_dtype)
            if x.numel():
                xs, ys = x.stride(), out.stride()
                _check(LIB.ttt_rope_apply(self._handle, B, H, N, x.data_ptr(), _strides(xs[0], xs[1], xs[2]),
                                          pos.data_ptr(), POS_DTYPE[pos.dtype], N * self.axes if pos.dim() == 3 else 0,
                                          out.data_ptr(), _strides(ys[0], ys[1], ys[2]), inverse, self._stream()),
                       "ttt_rope_apply")
        return out

    def forward(self, x, pos, out=None, stream=None):
        """x [B, H, N, d] (any strides, channels contiguous) turned to its positions pos [N, axes] or
        [B, N, axes], int32 or float32.  out: given, and then possibly x itself, or a new contiguous tensor."""
        return self._apply(x, pos, out, 0, stream, "x")

    def backward(self, dy, pos, out=None, stream=None):
        """The gradient of forward with respect to x: the rotation the other way."""
        return self._apply(dy, pos, out, 1, stream, "dy")


class GatedScan(_StatusOp):
    """Gated linear recurrence h_t = a_t h_{t-1} + u_t over [B, L, D].

    cfg: D, gate ("value": a = g, "sigmoid": a = sigma(g), "exp": a = exp(g)), inp ("plain": u = x,
    "complement": u = (1 - a) x), dtype ("bf16", "f32").  States (h0, h_last and their gradients) are fp32 [B, D].
    """

    def __post_init__(self):
        c, k = self.cfg, ScanConfig()
        k.D, k.gate, k.input, k.dtype = c["D"], GATE[c["gate"]], SCAN_INPUT[c["inp"]], DTYPE[c["dtype"]]
        self.D = int(c["D"])
        self._open(LIB.ttt_scan_create, LIB.ttt_scan_destroy, k)

    def _rows(self, B, L, **tensors):
        for name, t in tensors.items():
            if t is not None:
                self._tensor(name, t, (B, L, self.D), self.io_dtype)

    def _state(self, B, lengths, **tensors):
        for name, t in tensors.items():
            if t is not None:
                self._tensor(name, t, (B, self.D), torch.float32, rows=False)
        if lengths is not None:
            self._tensor("lengths", lengths, (B,), torch.int32, rows=False)

    def _shape(self, t, name):
        self._need_open()
        if t.dim() != 3 or t.shape[0] < 1:
            raise ValueError(f"{name}: expected [B, L, {self.D}], got shape {tuple(t.shape)}")
        return t.shape[0], t.shape[1]

    def _new(self, B, L, lengths, like):
        # rows behind a sequence's end are left as they are: zeros, in a tensor made here
        make = torch.empty if lengths is None else torch.zeros
        return make((B, L, self.D), dtype=self.io_dtype, device=like.device)

    def _workspace(self, B, L, like):
        n = LIB.ttt_scan_workspace_size(self._handle, B, L)
        return (torch.empty(n, dtype=torch.uint8, device=like.device), n) if n else (None, 0)

    def new_saved(self, B: int, L: int, stream=None):
        """A buffer for what a forward call leaves for its backward call."""
        self._need_open()
        with self._on(stream):
            return torch.empty(max(16, LIB.ttt_scan_saved_size(self._handle, B, L)), dtype=torch.uint8,
                               device=f"cuda:{self._index}")

    def _check_saved(self, saved, B, L):
        n = LIB.ttt_scan_saved_size(self._handle, B, L)
        if saved.dtype != torch.uint8 or saved.numel() < n or not saved.is_contiguous() or \
                saved.device.index != self._index:
            raise ValueError(f"saved: expected at least {n} contiguous bytes on cuda:{self._index} (new_saved)")

    def forward(self, g, x, h0=None, lengths=None, saved=None, out=None, h_last=None, stream=None):
        """Returns (h [B, L, D], h_last [B, D]).  lengths: [B] int32, each sequence's own length; rows from
        there on are not read and are left as they were in `out` (zero where it is not given).  h_last may be h0."""
        B, L = self._shape(x, "x")
        self._rows(B, L, g=g, x=x, out=out)
        self._state(B, lengths, h0=h0, h_last=h_last)
        if saved is not None:
            self._check_saved(saved, B, L)
        with self._on(stream, g, x, h0, lengths, saved, out, h_last):
            if out is None:
                out = self._new(B, L, lengths, x)
            if h_last is None:
                h_last = torch.empty((B, self.D), dtype=torch.float32, device=x.device)
            ws, n = self._workspace(B, L, x)
            gs, xs, hs = g.stride(), x.stride(), out.stride()
            _check(LIB.ttt_scan_forward(self._handle, B, L, g.data_ptr(), _strides(gs[0], 0, gs[1]), x.data_ptr(),
                                        _strides(xs[0], 0, xs[1]), _ptr(h0), _ptr(lengths), out.data_ptr(),
                                        _strides(hs[0], 0, hs[1]), h_last.data_ptr(), _ptr(saved), _ptr(ws), n,
                                        self._status.data_ptr(), self._stream()), "ttt_scan_forward")
        return out, h_last

    def backward(self, dh, g, x, saved, dh_last=None, lengths=None, dg=None, dx=None, dh0=None, stream=None):
        """Gradients (dg, dx [B, L, D], dh0 [B, D]) of a forward call with the same g, x and lengths that was
        given `saved`.  Rows behind a sequence's end are left as they were (zero in tensors made here)."""
        B, L = self._shape(x, "x")
        self._rows(B, L, dh=dh, g=g, x=x, dg=dg, dx=dx)
        self._state(B, lengths, dh_last=dh_last, dh0=dh0)
        self._check_saved(saved, B, L)
        with self._on(stream, dh, g, x, saved, dh_last, lengths, dg, dx, dh0):
            dg = self._new(B, L, lengths, x) if dg is None else dg
            dx = self._new(B, L, lengths, x) if dx is None else dx
            if dh0 is None:
                dh0 = torch.empty((B, self.D), dtype=torch.float32, device=x.device)
            ws, n = self._workspace(B, L, x)
            s = [_strides(t.stride(0), 0, t.stride(1)) for t in (dh, g, x, dg, dx)]
            _check(LIB.ttt_scan_backward(self._handle, B, L, dh.data_ptr(), s[0], _ptr(dh_last), g.data_ptr(), s[1],
                                         x.data_ptr(), s[2], _ptr(lengths), saved.data_ptr(), dg.data_ptr(), s[3],
                                         dx.data_ptr(), s[4], dh0.data_ptr(), _ptr(ws), n, self._status.data_ptr(),
                                         self._stream()), "ttt_scan_backward")
        return dg, dx, dh0


class GroupNorm(_StatusOp):
    """Group norm with an activation, channels last.

    cfg: C, groups, act ("none", "silu", "gelu"; default "none"), eps (default 1e-5), dtype ("bf16", "f32").
    x is [B, N, C], or [B, groups, N, C / groups] as TTTLayer returns it; y is [B, N, C].
    """

    def __post_init__(self):
        c, k = self.cfg, NormConfig()
        k.C, k.groups, k.act, k.eps = c["C"], c["groups"], ACT[c.get("act", "none")], c.get("eps", 1e-5)
        k.dtype = DTYPE[c["dtype"]]
        self.C, self.groups = int(c["C"]), int(c["groups"])
        self._open(LIB.ttt_norm_create, LIB.ttt_norm_destroy, k)

    def new_stats(self, B: int, stream=None):
        """A buffer for the mean and 1 / sqrt(var + eps) of every group, for the backward call."""
        self._need_open()
        with self._on(stream):
            return torch.empty((B, self.groups, 2), dtype=torch.float32, device=f"cuda:{self._index}")

    def _shape(self, x):
        self._need_open()
        n = self.C // self.groups
        if x.dim() == 4 and x.shape == (x.shape[0], self.groups, x.shape[2], n):
            B, N, shape = x.shape[0], x.shape[2], x.shape
        elif x.dim() == 3:
            B, N, shape = x.shape[0], x.shape[1], (x.shape[0], x.shape[1], self.C)
        else:
            raise ValueError(f"x: expected [B, N, {self.C}] or [B, {self.groups}, N, {n}], got {tuple(x.shape)}")
        if B < 1 or N < 1:
            raise ValueError(f"x: no statistics of an empty tensor, got shape {tuple(x.shape)}")
        return B, N, shape

    def _strides(self, t):
        s = t.stride()
        return _strides(s[0], self.C // self.groups, s[1]) if t.dim() == 3 else _strides(s[0], s[1], s[2])

    def _workspace(self, B, N, backward, like):
        n = LIB.ttt_norm_workspace_size(self._handle, B, N, backward)
        return (torch.empty(n, dtype=torch.uint8, device=like.device), n) if n else (None, 0)

    def _weights(self, **tensors):
        for name, t in tensors.items():
            if t is not None:
                self._tensor(name, t, (self.C,), torch.float32, rows=False)

    def forward(self, x, weight=None, bias=None, stats=None, out=None, stream=None):
        """y [B, N, C].  weight, bias: [C] fp32.  out: given, and then possibly x itself, or new."""
        B, N, shape = self._shape(x)
        self._tensor("x", x, shape, self.io_dtype)
        self._weights(weight=weight, bias=bias)
        if stats is not None:
            self._tensor("stats", stats, (B, self.groups, 2), torch.float32, rows=False)
        if out is not None:
            self._tensor("out", out, (B, N, self.C), self.io_dtype)
        with self._on(stream, x, weight, bias, stats, out):
            if out is None:
                out = torch.empty((B, N, self.C), dtype=self.io_dtype, device=x.device)
            ws, n = self._workspace(B, N, 0, x)
            _check(LIB.ttt_norm_forward(self._handle, B, N, x.data_ptr(), self._strides(x), _ptr(weight), _ptr(bias),
                                        out.data_ptr(), self._strides(out), _ptr(stats), _ptr(ws), n,
                                        self._status.data_ptr(), self._stream()), "ttt_norm_forward")
        return out

    def backward(self, dy, x, weight, bias, stats, dx=None, dweight=None, dbias=None, stream=None):
        """Gradients (dx of x's shape, dweight [C], dbias [C]) of a forward call that was given `stats`."""
        B, N, shape = self._shape(x)
        self._tensor("x", x, shape, self.io_dtype)
        self._tensor("dy", dy, (B, N, self.C), self.io_dtype)
        self._weights(weight=weight, bias=bias, dweight=dweight, dbias=dbias)
        self._tensor("stats", stats, (B, self.groups, 2), torch.float32, rows=False)
        if dx is not None:
            self._tensor("dx", dx, shape, self.io_dtype)
        with self._on(stream, dy, x, weight, bias, stats, dx, dweight, dbias):
            if dx is None:
                dx = torch.empty(shape, dtype=self.io_dtype, device=x.device)
            if dweight is None:
                dweight = torch.empty(self.C, dtype=torch.float32, device=x.device)
            if dbias is None:
                dbias = torch.empty(self.C, dtype=torch.float32, device=x.device)
            ws, n = self._workspace(B, N, 1, x)
            _check(LIB.ttt_norm_backward(self._handle, B, N, dy.data_ptr(), self._strides(dy), x.data_ptr(),
                                         self._strides(x), _ptr(weight), _ptr(bias), stats.data_ptr(), dx.data_ptr(),
                                         self._strides(dx), dweight.data_ptr(), dbias.data_ptr(), _ptr(ws), n,
                                         self._status.data_ptr(), self._stream()), "ttt_norm_backward")
        return dx, dweight, dbias
