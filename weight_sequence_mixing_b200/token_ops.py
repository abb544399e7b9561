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
from dataclasses import dataclass, field

import torch

from .binding import DTYPE, LIB, TTT_ERR_CUDA, TTT_ERR_TIMEOUT, _check

# what a call of a few microseconds can afford of torch: no stream or device objects
_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream

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


class _Strides(dict):
    """ttt_strides by a tensor's strides (kept: a program has few, and a call needs several)."""

    def __init__(self, convert):
        super().__init__()
        self._convert = convert

    def __missing__(self, key):
        if len(self) >= 4096:
            self.clear()
        s = self[key] = (ctypes.c_int64 * 3)(*self._convert(*key))
        return s


_HEADS = _Strides(lambda batch, head, token, _: (batch, head, token))
_ROWS = _Strides(lambda batch, token, _: (batch, 0, token))


def _ptr(t):
    return None if t is None else t.data_ptr()


def _plain(x, shape, dtype):
    """A new contiguous tensor on x's device (the first form takes half the second's time)."""
    if x.shape == shape and x.dtype == dtype and x.is_contiguous():
        return torch.empty_like(x)
    return x.new_empty(shape, dtype=dtype)


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
        self._handle, self._destroy = h, destroy
        self.io_dtype = torch.float32 if self.cfg["dtype"] == "f32" else torch.bfloat16
        dev = torch.device(self.device)
        if dev.type != "cuda":
            raise ValueError(f"device: expected a CUDA device, got {self.device}")
        self._index = dev.index
        if self._index is None:
            self._index = torch.cuda.current_device() if torch.cuda.is_available() else 0

    def close(self):
        if self._handle:
            self._destroy(self._handle)
            self._handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _open_handle(self):
        if not self._handle:
            raise ValueError(f"{type(self).__name__} is closed")
        return self._handle

    def _rows(self, name, t, shape, dtype):
        """`t` is on this device, of this shape and type, and its rows are contiguous."""
        if t.dtype == dtype and t.shape == shape and t.get_device() == self._index and t.stride()[-1] == 1:
            return
        if t.dtype != dtype or t.shape != shape:
            raise ValueError(f"{name}: expected shape {tuple(shape)} of {dtype}, got {tuple(t.shape)} of {t.dtype}")
        if t.get_device() != self._index:
            raise ValueError(f"{name}: expected a tensor on cuda:{self._index}, got one on {t.device}")
        if t.stride(-1) != 1 and shape[-1] > 1:
            raise ValueError(f"{name}: the channels of a row must be contiguous, got strides {t.stride()}")

    def _whole(self, name, t, shape, dtype):
        """`t` is on this device, of this shape and type, and contiguous."""
        if t.dtype == dtype and t.shape == shape and t.get_device() == self._index and t.is_contiguous():
            return
        self._rows(name, t, shape, dtype)
        if not t.is_contiguous():
            raise ValueError(f"{name}: must be contiguous, got strides {t.stride()}")

    def _run(self, stream, tensors, call, *args):
        """call(*args) with this device current, on `stream` or the current stream.  Tensors handed to
        another stream than the current one are kept from reuse until that stream is done with them."""
        if stream is None:
            if _current_device() == self._index:
                return call(*args)
            with torch.cuda.device(self._index):
                return call(*args)
        if stream.device.index != self._index:
            raise ValueError(f"stream: expected one of cuda:{self._index}, got one of {stream.device}")
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
        with torch.cuda.stream(stream):
            return call(*args)


class _Sizes(dict):
    """Byte counts that depend on a call's sizes alone, asked of the library once for each."""

    def __init__(self, ask):
        super().__init__()
        self._ask = ask

    def __missing__(self, key):
        if len(self) >= 4096:
            self.clear()
        n = self[key] = self._ask(*key)
        return n


class _StatusOp(_Op):
    """An operator whose kernels wait on one another and report a wait that ran out."""

    def _open(self, create, destroy, config):
        super()._open(create, destroy, config)
        self._status = torch.zeros(1, dtype=torch.int32, device=f"cuda:{self._index}")
        self._status_ptr = self._status.data_ptr()

    def _bytes(self, n):
        """n bytes of workspace, or none."""
        return torch.empty(n, dtype=torch.uint8, device=self._status.device) if n else None

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
        self.d, self.axes = int(c["d"]), len(pairs)
        self._open(LIB.ttt_rope_create, LIB.ttt_rope_destroy, k)

    def _apply(self, name, x, pos, out, stream, inverse):
        shape = x.shape
        if len(shape) != 4:
            raise ValueError(f"{name}: expected [B, H, N, {self.d}], got shape {tuple(shape)}")
        B, H, N, _ = shape
        self._rows(name, x, (B, H, N, self.d), self.io_dtype)
        kind = POS_DTYPE.get(pos.dtype)
        each = len(pos.shape) == 3
        if kind is None or pos.shape != ((B, N, self.axes) if each else (N, self.axes)):
            raise ValueError(f"pos: expected [{N}, {self.axes}] or [{B}, {N}, {self.axes}] of int32 or float32, got "
                             f"shape {tuple(pos.shape)} of {pos.dtype}")
        if not pos.is_contiguous() or pos.get_device() != self._index:
            self._whole("pos", pos, pos.shape, pos.dtype)
        if out is not None:
            self._rows("out", out, shape, self.io_dtype)
        return self._run(stream, (x, pos, out), self._launch, self._open_handle(), x, pos, out, kind, each, inverse)

    def _launch(self, handle, x, pos, out, kind, each, inverse):
        shape = x.shape
        if out is None:
            out = _plain(x, shape, self.io_dtype)
        B, H, N, _ = shape
        if B and H and N:
            st = LIB.ttt_rope_apply(handle, B, H, N, x.data_ptr(), _HEADS[x.stride()], pos.data_ptr(), kind,
                                    N * self.axes if each else 0, out.data_ptr(), _HEADS[out.stride()], inverse,
                                    _current_stream(self._index))
            if st:
                _check(st, "ttt_rope_apply")
        return out

    def forward(self, x, pos, out=None, stream=None):
        """x [B, H, N, d] (any strides, channels contiguous) turned to its positions pos [N, axes] or
        [B, N, axes], int32 or float32.  out: given, and then possibly x itself, or a new contiguous tensor."""
        return self._apply("x", x, pos, out, stream, 0)

    def backward(self, dy, pos, out=None, stream=None):
        """The gradient of forward with respect to x: the rotation the other way."""
        return self._apply("dy", dy, pos, out, stream, 1)


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
        self._space = _Sizes(lambda B, L: LIB.ttt_scan_workspace_size(self._handle, B, L))
        self._saved = _Sizes(lambda B, L: LIB.ttt_scan_saved_size(self._handle, B, L))

    def _sizes(self, x, lengths):
        shape = x.shape
        if len(shape) != 3 or shape[0] < 1:
            raise ValueError(f"x: expected [B, L, {self.D}], got shape {tuple(shape)}")
        if lengths is not None:
            self._whole("lengths", lengths, (shape[0],), torch.int32)
        return (shape[0], shape[1], self.D), (shape[0], self.D)

    def _check_saved(self, saved, B, L):
        n = self._saved[B, L]
        if saved.dtype != torch.uint8 or saved.numel() < n or not saved.is_contiguous() or \
                saved.get_device() != self._index:
            raise ValueError(f"saved: expected at least {n} contiguous bytes on cuda:{self._index} (new_saved)")

    def new_saved(self, B: int, L: int, stream=None):
        """A buffer for what a forward call leaves for its backward call."""
        self._open_handle()
        return self._run(stream, (), self._bytes, max(16, self._saved[B, L]))

    def _new(self, handle, x, shape, lengths):
        out = _plain(x, shape, self.io_dtype)
        if lengths is not None:  # rows behind a sequence's end are left as they are: zeros, in a tensor made here
            st = LIB.ttt_scan_clear(handle, shape[0], shape[1], lengths.data_ptr(), out.data_ptr(), _ROWS[out.stride()],
                                    _current_stream(self._index))
            if st:
                _check(st, "ttt_scan_clear")
        return out

    def forward(self, g, x, h0=None, lengths=None, saved=None, out=None, h_last=None, stream=None):
        """Returns (h [B, L, D], h_last [B, D]).  lengths: [B] int32, each sequence's own length; rows from
        there on are not used and are left as they were in `out` (zero where it is not given).  h_last may be h0."""
        shape, state = self._sizes(x, lengths)
        self._rows("x", x, shape, self.io_dtype)
        self._rows("g", g, shape, self.io_dtype)
        if out is not None:
            self._rows("out", out, shape, self.io_dtype)
        if h0 is not None:
            self._whole("h0", h0, state, torch.float32)
        if h_last is not None:
            self._whole("h_last", h_last, state, torch.float32)
        if saved is not None:
            self._check_saved(saved, shape[0], shape[1])
        return self._run(stream, (g, x, h0, lengths, saved, out, h_last), self._launch_forward, self._open_handle(), g, x,
                         h0, lengths, saved, out, h_last, shape, state)

    def _launch_forward(self, handle, g, x, h0, lengths, saved, out, h_last, shape, state):
        B, L, _ = shape
        if out is None:
            out = self._new(handle, x, shape, lengths)
        if h_last is None:
            h_last = _plain(x if h0 is None else h0, state, torch.float32)
        n = self._space[B, L]
        ws = self._bytes(n)
        st = LIB.ttt_scan_forward(handle, B, L, g.data_ptr(), _ROWS[g.stride()], x.data_ptr(), _ROWS[x.stride()], _ptr(h0),
                                  _ptr(lengths), out.data_ptr(), _ROWS[out.stride()], h_last.data_ptr(), _ptr(saved),
                                  _ptr(ws), n, self._status_ptr, _current_stream(self._index))
        if st:
            _check(st, "ttt_scan_forward")
        return out, h_last

    def backward(self, dh, g, x, saved, dh_last=None, lengths=None, dg=None, dx=None, dh0=None, stream=None):
        """Gradients (dg, dx [B, L, D], dh0 [B, D]) of a forward call with the same g, x and lengths that was
        given `saved`.  Rows behind a sequence's end are left as they were (zero in tensors made here)."""
        shape, state = self._sizes(x, lengths)
        for name, t in (("x", x), ("g", g), ("dh", dh), ("dg", dg), ("dx", dx)):
            if t is not None:
                self._rows(name, t, shape, self.io_dtype)
        for name, t in (("dh_last", dh_last), ("dh0", dh0)):
            if t is not None:
                self._whole(name, t, state, torch.float32)
        self._check_saved(saved, shape[0], shape[1])
        return self._run(stream, (dh, g, x, saved, dh_last, lengths, dg, dx, dh0), self._launch_backward,
                         self._open_handle(), dh, g, x, saved, dh_last, lengths, dg, dx, dh0, shape, state)

    def _launch_backward(self, handle, dh, g, x, saved, dh_last, lengths, dg, dx, dh0, shape, state):
        B, L, _ = shape
        dg = self._new(handle, x, shape, lengths) if dg is None else dg
        dx = self._new(handle, x, shape, lengths) if dx is None else dx
        if dh0 is None:
            dh0 = _plain(x if dh_last is None else dh_last, state, torch.float32)
        n = self._space[B, L]
        ws = self._bytes(n)
        st = LIB.ttt_scan_backward(handle, B, L, dh.data_ptr(), _ROWS[dh.stride()], _ptr(dh_last), g.data_ptr(),
                                   _ROWS[g.stride()], x.data_ptr(), _ROWS[x.stride()], _ptr(lengths), saved.data_ptr(),
                                   dg.data_ptr(), _ROWS[dg.stride()], dx.data_ptr(), _ROWS[dx.stride()], dh0.data_ptr(),
                                   _ptr(ws), n, self._status_ptr, _current_stream(self._index))
        if st:
            _check(st, "ttt_scan_backward")
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
        self._open(LIB.ttt_norm_create, LIB.ttt_norm_destroy, k)
        self.C, self.groups = int(c["C"]), int(c["groups"])
        self._space = _Sizes(lambda B, N, backward: LIB.ttt_norm_workspace_size(self._handle, B, N, backward))
        each = self._each = self.C // self.groups  # channels of a group
        self._channels_last = _Strides(lambda batch, token, _: (batch, each, token))

    def new_stats(self, B: int, stream=None):
        """A buffer for the mean and 1 / sqrt(var + eps) of every group, for the backward call."""
        self._open_handle()
        return self._run(stream, (), _plain, self._status.view(torch.float32), (B, self.groups, 2), torch.float32)

    def _shapes(self, x):
        """(shape x has to have, [B, N, C])"""
        s = x.shape
        if len(s) == 3:
            want = rows = (s[0], s[1], self.C)
        elif len(s) == 4:
            want, rows = (s[0], self.groups, s[2], self._each), (s[0], s[2], self.C)
        else:
            raise ValueError(f"x: expected [B, N, {self.C}] or [B, {self.groups}, N, {self._each}], got {tuple(s)}")
        if s[0] < 1 or rows[1] < 1:
            raise ValueError(f"x: no statistics of an empty tensor, got shape {tuple(s)}")
        return want, rows

    def _by_group(self, t):
        s = t.stride()
        return self._channels_last[s] if len(s) == 3 else _HEADS[s]

    def forward(self, x, weight=None, bias=None, stats=None, out=None, stream=None):
        """y [B, N, C].  weight, bias: [C] fp32.  out: given, and then possibly x itself, or new."""
        want, rows = self._shapes(x)
        self._rows("x", x, want, self.io_dtype)
        if weight is not None:
            self._whole("weight", weight, (self.C,), torch.float32)
        if bias is not None:
            self._whole("bias", bias, (self.C,), torch.float32)
        if stats is not None:
            self._whole("stats", stats, (rows[0], self.groups, 2), torch.float32)
        if out is not None:
            self._rows("out", out, rows, self.io_dtype)
        return self._run(stream, (x, weight, bias, stats, out), self._launch_forward, self._open_handle(), x, weight, bias,
                         stats, out, rows)

    def _launch_forward(self, handle, x, weight, bias, stats, out, rows):
        if out is None:
            out = _plain(x, rows, self.io_dtype)
        n = self._space[rows[0], rows[1], 0]
        ws = self._bytes(n)
        st = LIB.ttt_norm_forward(handle, rows[0], rows[1], x.data_ptr(), self._by_group(x), _ptr(weight), _ptr(bias),
                                  out.data_ptr(), self._channels_last[out.stride()], _ptr(stats), _ptr(ws), n, self._status_ptr,
                                  _current_stream(self._index))
        if st:
            _check(st, "ttt_norm_forward")
        return out

    def backward(self, dy, x, weight, bias, stats, dx=None, dweight=None, dbias=None, stream=None):
        """Gradients (dx of x's shape, dweight [C], dbias [C]) of a forward call that was given `stats`."""
        want, rows = self._shapes(x)
        self._rows("x", x, want, self.io_dtype)
        self._rows("dy", dy, rows, self.io_dtype)
        for name, t in (("weight", weight), ("bias", bias), ("dweight", dweight), ("dbias", dbias)):
            if t is not None:
                self._whole(name, t, (self.C,), torch.float32)
        self._whole("stats", stats, (rows[0], self.groups, 2), torch.float32)
        if dx is not None:
            self._rows("dx", dx, want, self.io_dtype)
        return self._run(stream, (dy, x, weight, bias, stats, dx, dweight, dbias), self._launch_backward,
                         self._open_handle(), dy, x, weight, bias, stats, dx, dweight, dbias, want, rows)

    def _launch_backward(self, handle, dy, x, weight, bias, stats, dx, dweight, dbias, want, rows):
        if dx is None:
            dx = _plain(x, want, self.io_dtype)
        if dweight is None:
            dweight = _plain(x if weight is None else weight, (self.C,), torch.float32)
        if dbias is None:
            dbias = _plain(x if bias is None else bias, (self.C,), torch.float32)
        n = self._space[rows[0], rows[1], 1]
        ws = self._bytes(n)
        st = LIB.ttt_norm_backward(handle, rows[0], rows[1], dy.data_ptr(), self._channels_last[dy.stride()], x.data_ptr(),
                                   self._by_group(x), _ptr(weight), _ptr(bias), stats.data_ptr(), dx.data_ptr(),
                                   self._by_group(dx), dweight.data_ptr(), dbias.data_ptr(), _ptr(ws), n,
                                   self._status_ptr, _current_stream(self._index))
        if st:
            _check(st, "ttt_norm_backward")
        return dx, dweight, dbias
