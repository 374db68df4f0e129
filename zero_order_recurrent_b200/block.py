"""Binding of the selective state-space block's operators (C ABI in include/zo_block.h).

Argument marshalling only, as in the package's other calls: outputs are the
caller's tensors, work is enqueued on the current torch stream of the tensors'
device (or on `stream`), and non-zero status codes become ZOError.  Tensors are
checked against one another here, where their types and shapes are known
(ValueError), sizes and pointers by the library.

Shapes: activations [rows, seq, channels] ([rows, channels] for single tokens and
norms) in float32, bfloat16 or float16 with any strides whose innermost is 1;
parameters float32, with or without a leading dimension of parameter sets (rows
are divided evenly among the sets, in order); recurrent states float32 (the
convolution's window has the activations' type).  `lengths` is int32 [rows].
Where `workspace` is not given, it comes from torch's allocator for this call.
"""
from __future__ import annotations

import ctypes
import struct

from . import ZO_DTYPE_BF16, ZO_DTYPE_FP32, _check, load_library

ZO_DTYPE_FP16 = 2
ZO_MAX_TAPS = 8
ZO_MAX_STATES = 128
ZO_MAX_NORM_WIDTH = 16384
ZO_CONV_SILU = 1
ZO_SCAN_SOFTPLUS = 1
ZO_SCAN_CHUNK = 16
ZO_NORM_GATE_FIRST = 1

_P, _I32, _I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class _Tensor(ctypes.Structure):
    _fields_ = [("ptr", _P), ("row", _I64), ("step", _I64)]


class _F32(ctypes.Structure):
    _fields_ = [("ptr", _P), ("stride", _I64)]


class ConvArgs(ctypes.Structure):
    _fields_ = [(n, _I32) for n in ("rows", "seq", "channels", "taps", "sets", "dtype", "flags")] + [
        ("x", _Tensor), ("out", _Tensor), ("weight", _F32), ("bias", _F32), ("lengths", _P),
        ("state_in", _Tensor), ("state_out", _Tensor), ("status", _P)]


class ConvGrads(ctypes.Structure):
    _fields_ = [("dout", _Tensor), ("dx", _Tensor), ("dweight", _F32), ("dbias", _F32),
                ("dstate_out", _Tensor), ("dstate_in", _Tensor)]


class ScanArgs(ctypes.Structure):
    _fields_ = [(n, _I32) for n in ("rows", "seq", "channels", "groups", "states", "sets", "dtype",
                                    "flags")] + [
        (n, _Tensor) for n in ("u", "delta", "out", "z", "B", "C")] + [
        (n, _F32) for n in ("A", "skip", "delta_bias")] + [
        ("lengths", _P), ("state_in", _F32), ("state_out", _F32), ("checkpoints", _P),
        ("status", _P)]


class ScanGrads(ctypes.Structure):
    _fields_ = [(n, _Tensor) for n in ("dout", "du", "ddelta", "dz", "dB", "dC")] + [
        (n, _F32) for n in ("dA", "dskip", "ddelta_bias", "dstate_out", "dstate_in")]


class NormArgs(ctypes.Structure):
    _fields_ = [(n, _I32) for n in ("rows", "channels", "sets", "dtype", "x_dtype", "flags")] + [
        ("eps", ctypes.c_float)] + [(n, _Tensor) for n in ("x", "x_out", "o", "gate", "n_out")] + [
        (n, _F32) for n in ("w_post", "scale", "w_pre")]


class NormGrads(ctypes.Structure):
    _fields_ = [(n, _Tensor) for n in ("dn", "dx_out", "dx", "d_o", "dgate")] + [
        (n, _F32) for n in ("dw_post", "dscale", "dw_pre")]


def declare(lib):
    """Declare the signatures of include/zo_block.h on the loaded library."""
    A = ctypes.POINTER
    sig = {
        "zo_conv": ([A(ConvArgs), _P], ctypes.c_int),
        "zo_conv_step": ([A(ConvArgs), _P], ctypes.c_int),
        "zo_conv_backward_workspace": ([A(ConvArgs)], _I64),
        "zo_conv_backward": ([A(ConvArgs), A(ConvGrads), _P, _I64, _P], ctypes.c_int),
        "zo_scan_workspace": ([A(ScanArgs)], _I64),
        "zo_scan_backward_workspace": ([A(ScanArgs)], _I64),
        "zo_scan": ([A(ScanArgs), _P, _I64, _P], ctypes.c_int),
        "zo_scan_step": ([A(ScanArgs), _P], ctypes.c_int),
        "zo_scan_backward": ([A(ScanArgs), A(ScanGrads), _P, _I64, _P], ctypes.c_int),
        "zo_block_norm": ([A(NormArgs), _P], ctypes.c_int),
        "zo_block_norm_backward_workspace": ([A(NormArgs)], _I64),
        "zo_block_norm_backward": ([A(NormArgs), A(NormGrads), _P, _I64, _P], ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res


torch = None   # imported by the first call, as by the package's other calls
_DTYPES = {}


def _import_torch():
    global torch
    import torch
    _DTYPES.update({torch.float32: ZO_DTYPE_FP32, torch.bfloat16: ZO_DTYPE_BF16,
                    torch.float16: ZO_DTYPE_FP16})


def _packer(structure):
    """struct.Struct with the layout of a ctypes Structure, its parts spelled out flat: packing
    one is several times quicker than filling the nested fields of the other."""
    code = {_I32: "i", ctypes.c_float: "f", _P: "P", _I64: "q"}

    def flat(s):
        for _, t in s._fields_:
            if hasattr(t, "_fields_"):
                yield from flat(t)
            else:
                yield code[t]
    p = struct.Struct("@" + "".join(flat(structure)))
    assert p.size == ctypes.sizeof(structure)
    return p.pack


_PACK = {t: _packer(t) for t in (ConvArgs, ConvGrads, ScanArgs, ScanGrads, NormArgs, NormGrads)}
_CALLS = {}  # the library's functions, taking packed structures
_NONE2, _NONE3 = (0, 0), (0, 0, 0)


class _Call:
    """The tensors of one call: checks them against the first one's device.  act, param, grad and
    states give a tensor's fields of the C structures."""

    def __init__(self, where, first):
        if torch is None:
            _import_torch()
        if not isinstance(first, torch.Tensor) or not first.is_cuda:
            raise ValueError(f"{where}: CUDA tensors are required")
        self.where = where
        self.index = first.get_device()

    def fail(self, name, what):
        raise ValueError(f"{self.where}: {name} {what}")

    def check(self, name, t, dtype):
        if not isinstance(t, torch.Tensor) or t.get_device() != self.index:
            self.fail(name, f"must be a tensor on cuda:{self.index}")
        if t.dtype is not dtype:
            self.fail(name, f"must be {dtype}, got {t.dtype}")

    def code(self, t):
        c = _DTYPES.get(t.dtype)
        if c is None:
            raise ValueError(f"{self.where}: float32, bfloat16 or float16 is required, "
                             f"got {t.dtype}")
        return c

    def act(self, name, t, shape, dtype, optional=False, inner=1):
        """A tensor of this shape: rows, steps or none, and `inner` contiguous dimensions."""
        if t is None and optional:
            return _NONE3
        if t is None or t.dtype is not dtype or t.get_device() != self.index:
            self.check(name, t, dtype)
        if t.shape != shape:
            self.fail(name, f"must have shape {tuple(shape)}, got {tuple(t.shape)}")
        st = t.stride()
        if st[-1] != 1 and shape[-1] != 1:
            self.fail(name, "must be contiguous in its last dimension")
        if inner == 2 and st[-2] != shape[-1] and shape[-2] != 1:
            self.fail(name, "must be contiguous in its last two dimensions")
        return t.data_ptr(), st[0], st[1] if len(st) - inner == 2 else 0

    def param(self, name, t, inner, sets, optional=False):
        """Parameters [inner] or [sets, inner]."""
        if t is None and optional:
            return _NONE2
        if t is None or t.dtype is not torch.float32 or t.get_device() != self.index:
            self.check(name, t, torch.float32)
        n, shape = len(inner), t.shape
        if shape[-n:] != inner or len(shape) - n not in (0, 1):
            self.fail(name, f"must have shape {tuple(inner)} or [sets, ...], got {tuple(shape)}")
        st = self.contiguous(name, t, n)
        if len(shape) == n or shape[0] == 1:
            return t.data_ptr(), 0
        if shape[0] != sets:
            self.fail(name, f"has {shape[0]} sets, others {sets}")
        return t.data_ptr(), st[0]

    def contiguous(self, name, t, n):
        """The strides of a tensor whose last n dimensions are contiguous."""
        st = t.stride()
        if not t.is_contiguous():
            want = 1
            for size, stride in zip(reversed(t.shape[-n:]), reversed(st[-n:])):
                if size != 1 and stride != want:
                    self.fail(name, f"must be contiguous in its last {n} dimensions")
                want *= size
        return st

    def grad(self, name, t, inner, sets, optional=False):
        """Parameter gradients: one for each set."""
        if t is None and optional:
            return _NONE2
        if t is None or t.dtype is not torch.float32 or t.get_device() != self.index:
            self.check(name, t, torch.float32)
        n = len(inner)
        if not (t.shape == (sets, *inner) or (sets == 1 and t.shape == inner)):
            self.fail(name, f"must have shape {(sets, *inner)}, got {tuple(t.shape)}")
        st = self.contiguous(name, t, n)
        return t.data_ptr(), st[0] if len(st) > n else 0

    def states(self, name, t, shape, optional=True):
        """Recurrent states [rows, channels, states]."""
        if t is None and optional:
            return _NONE2
        if t is None or t.dtype is not torch.float32 or t.get_device() != self.index:
            self.check(name, t, torch.float32)
        if t.shape != shape:
            self.fail(name, f"must have shape {tuple(shape)}, got {tuple(t.shape)}")
        return t.data_ptr(), self.contiguous(name, t, 2)[0]

    def ints(self, name, t, n):
        if t is None:
            return 0
        self.check(name, t, torch.int32)
        if t.shape != (n,) or (n != 1 and t.stride(0) != 1):
            self.fail(name, f"must be contiguous of shape {(n,)}")
        return t.data_ptr()

    def pack(self, structure, values):
        try:
            return _PACK[structure](*values)
        except (struct.error, OverflowError, TypeError) as e:
            raise ValueError(f"{self.where}: a size or eps does not fit the call ({e})") from None

    def run(self, name, *args, stream=None, workspace=None):
        """Calls `name` on the tensors' device.  workspace: None for a call without
        one, else (the caller's tensor or None, bytes)."""
        cur = torch.cuda.current_stream(self.index)
        handle = current = cur.cuda_stream
        if stream is not None:
            handle = stream if isinstance(stream, int) else stream.cuda_stream
        if workspace is not None:
            ws, need = workspace
            if need < 0:
                # the sizes are refused: the call itself says why
                args += (None, 0)
            elif ws is None:
                if need:
                    ws = torch.empty(need, dtype=torch.uint8, device=f"cuda:{self.index}")
                    if handle != current:
                        # the allocator would hand it out again on the current stream
                        other = stream if not isinstance(stream, int) else \
                            torch.cuda.ExternalStream(stream, device=self.index)
                        other.wait_stream(cur)
                        ws.record_stream(other)
                args += (ws.data_ptr() if need else None, need)
            else:
                if not isinstance(ws, torch.Tensor) or ws.get_device() != self.index or \
                        not ws.is_contiguous():
                    self.fail("workspace", f"must be a contiguous tensor on cuda:{self.index}")
                args += (ws.data_ptr(), ws.numel() * ws.element_size())
        f = _call(name)
        if torch.cuda.current_device() == self.index:
            st = f(*args, handle)
        else:
            with torch.cuda.device(self.index):
                st = f(*args, handle)
        if st:
            _check(st, name)


def _call(name):
    f = _CALLS.get(name)
    if f is None:
        of = getattr(load_library(), name)
        types = [_P if hasattr(t, "contents") else t for t in of.argtypes]
        f = _CALLS[name] = ctypes.CFUNCTYPE(of.restype, *types)((name, load_library()))
    return f


def _sets(*pairs):
    """The number of parameter sets of (tensor, inner dimensions) pairs."""
    s = 1
    for t, n in pairs:
        if t is not None and t.dim() == n + 1 and t.shape[0] > s:
            s = t.shape[0]
    return s


# ---- short causal convolution ----------------------------------------------------

def _conv_args(c, x, weight, out, bias, silu, lengths, state_in, state_out, status):
    if x.dim() not in (2, 3) or weight.dim() not in (2, 3):
        c.fail("x, weight", "must be [rows, seq, channels] and [taps, channels]")
    dt = x.dtype
    R, D = x.shape[0], x.shape[-1]
    T = x.shape[1] if x.dim() == 3 else 1
    K = weight.shape[-2]
    S = _sets((weight, 2), (bias, 1))
    win = (R, K - 1, D)
    # a window of one tap holds nothing
    st = [_NONE3 if K == 1 else c.act(n, t, win, dt, True)
          for n, t in (("state_in", state_in), ("state_out", state_out))]
    args = (
        R, T, D, K, S, c.code(x), ZO_CONV_SILU if silu else 0, *c.act("x", x, x.shape, dt),
        *c.act("out", out, x.shape, dt, True), *c.param("weight", weight, (K, D), S),
        *c.param("bias", bias, (D,), S, True), c.ints("lengths", lengths, R), *st[0], *st[1],
        c.ints("status", status, 1))
    return (K, S), c.pack(ConvArgs, args)


def zo_conv(x, weight, out, bias=None, silu=True, lengths=None, state_in=None, state_out=None,
            status=None, stream=None):
    """Short causal convolution of whole rows: out_t = silu(bias + sum_k weight[k] x_{t-taps+1+k}).

    x, out [rows, seq, channels]; weight [taps, channels] or [sets, taps, channels];
    state_in/state_out [rows, taps-1, channels]: the inputs before the first step and before
    the row's end (state_out may be state_in).  Steps from a row's length on give 0."""
    c = _Call("zo_conv", x)
    if x.dim() != 3:
        c.fail("x", "must be [rows, seq, channels]")
    _, a = _conv_args(c, x, weight, out, bias, silu, lengths, state_in, state_out, status)
    c.run("zo_conv", a, stream=stream)


def zo_conv_step(x, weight, state, out, bias=None, silu=True, state_out=None, stream=None):
    """One step of zo_conv: x, out [rows, channels], state [rows, taps-1, channels].

    The moved window is written to state_out (default: state itself)."""
    c = _Call("zo_conv_step", x)
    if x.dim() != 2:
        c.fail("x", "must be [rows, channels]")
    _, a = _conv_args(c, x, weight, out, bias, silu, None, state,
                      state if state_out is None else state_out, None)
    c.run("zo_conv_step", a, stream=stream)


def zo_conv_backward(x, weight, dout, dx, dweight, bias=None, dbias=None, silu=True, lengths=None,
                     state_in=None, dstate_out=None, dstate_in=None, workspace=None, stream=None):
    """Gradients of zo_conv from dout: dx (0 from a row's length on), dweight [sets, taps,
    channels], and where given dbias, dstate_in (of state_in)."""
    c = _Call("zo_conv_backward", x)
    if x.dim() != 3:
        c.fail("x", "must be [rows, seq, channels]")
    (K, S), a = _conv_args(c, x, weight, None, bias, silu, lengths, state_in, None, None)
    dt, (R, _, D) = x.dtype, x.shape
    st = [_NONE3 if K == 1 else c.act(n, t, (R, K - 1, D), dt, True)
          for n, t in (("dstate_out", dstate_out), ("dstate_in", dstate_in))]
    g = _PACK[ConvGrads](*c.act("dout", dout, x.shape, dt), *c.act("dx", dx, x.shape, dt),
                         *c.grad("dweight", dweight, (K, D), S),
                         *c.grad("dbias", dbias, (D,), S, True), *st[0], *st[1])
    need = _call("zo_conv_backward_workspace")(a)
    c.run("zo_conv_backward", a, g, stream=stream, workspace=(workspace, need))


# ---- selective scan ----------------------------------------------------------------

def zo_scan_checkpoint_shape(shape, states):
    """Shape of zo_scan's checkpoints (float32) for u of `shape` [rows, seq, channels]."""
    R, T, D = shape
    return (R, -(-T // ZO_SCAN_CHUNK), D, states)


def _scan_args(c, u, delta, A, B, C, out, skip, z, delta_bias, softplus, lengths, state_in,
               state_out, checkpoints, status):
    dt = u.dtype
    if u.dim() not in (2, 3) or A.dim() not in (2, 3) or B.dim() != u.dim() + 1:
        c.fail("u, A, B", "must be [rows, seq, channels], [channels, states] and "
                          "[rows, seq, groups, states]")
    R, D = u.shape[0], u.shape[-1]
    T = u.shape[1] if u.dim() == 3 else 1
    G, N = B.shape[-2:]
    S = _sets((A, 2), (skip, 1), (delta_bias, 1))
    shp = (*u.shape[:-1], G, N)
    kept = 0
    if checkpoints is not None:
        c.check("checkpoints", checkpoints, torch.float32)
        if checkpoints.shape != (R, -(-T // ZO_SCAN_CHUNK), D, N) or \
                not checkpoints.is_contiguous():
            c.fail("checkpoints", "must be contiguous of zo_scan_checkpoint_shape()")
        kept = checkpoints.data_ptr()
    args = (
        R, T, D, G, N, S, c.code(u), ZO_SCAN_SOFTPLUS if softplus else 0,
        *c.act("u", u, u.shape, dt), *c.act("delta", delta, u.shape, dt),
        *c.act("out", out, u.shape, dt, True), *c.act("z", z, u.shape, dt, True),
        *c.act("B", B, shp, dt, inner=2), *c.act("C", C, shp, dt, inner=2),
        *c.param("A", A, (D, N), S), *c.param("skip", skip, (D,), S, True),
        *c.param("delta_bias", delta_bias, (D,), S, True), c.ints("lengths", lengths, R),
        *c.states("state_in", state_in, (R, D, N)), *c.states("state_out", state_out, (R, D, N)),
        kept, c.ints("status", status, 1))
    return (N, S), c.pack(ScanArgs, args)


def zo_scan(u, delta, A, B, C, out, skip=None, z=None, delta_bias=None, softplus=True,
            lengths=None, state_in=None, state_out=None, checkpoints=None, workspace=None,
            status=None, stream=None):
    """Selective scan of whole rows (include/zo_block.h has the formulas).

    u, delta, z, out [rows, seq, channels]; B, C [rows, seq, groups, states]; A [channels,
    states] or [sets, channels, states]; skip, delta_bias [channels] or [sets, channels];
    state_in/state_out [rows, channels, states].  For zo_scan_backward give checkpoints of
    zo_scan_checkpoint_shape().  Steps from a row's length on give 0."""
    c = _Call("zo_scan", u)
    if u.dim() != 3:
        c.fail("u", "must be [rows, seq, channels]")
    _, a = _scan_args(c, u, delta, A, B, C, out, skip, z, delta_bias, softplus, lengths, state_in,
                      state_out, checkpoints, status)
    need = _call("zo_scan_workspace")(a)
    c.run("zo_scan", a, stream=stream, workspace=(workspace, need))


def zo_scan_step(u, delta, A, B, C, state, out, skip=None, z=None, delta_bias=None, softplus=True,
                 state_out=None, stream=None):
    """One step of zo_scan: u, delta, z, out [rows, channels]; B, C [rows, groups, states].

    The new state is written to state_out (default: state itself)."""
    c = _Call("zo_scan_step", u)
    if u.dim() != 2:
        c.fail("u", "must be [rows, channels]")
    _, a = _scan_args(c, u, delta, A, B, C, out, skip, z, delta_bias, softplus, None, state,
                      state if state_out is None else state_out, None, None)
    c.run("zo_scan_step", a, stream=stream)


def zo_scan_backward(u, delta, A, B, C, dout, checkpoints, du, ddelta, dA, dB, dC, skip=None,
                     dskip=None, z=None, dz=None, delta_bias=None, ddelta_bias=None, softplus=True,
                     lengths=None, dstate_out=None, dstate_in=None, workspace=None, stream=None):
    """Gradients of zo_scan from dout and the checkpoints that zo_scan wrote for the same inputs.

    Gradients have the shapes of what they belong to; those of parameters [sets, ...].  dskip,
    ddelta_bias, dstate_in (of state_in) are written where given; dz is required with z."""
    c = _Call("zo_scan_backward", u)
    if u.dim() != 3:
        c.fail("u", "must be [rows, seq, channels]")
    (N, S), a = _scan_args(c, u, delta, A, B, C, None, skip, z, delta_bias, softplus, lengths,
                           None, None, checkpoints, None)
    dt, (R, _, D) = u.dtype, u.shape
    g = _PACK[ScanGrads](
        *c.act("dout", dout, u.shape, dt), *c.act("du", du, u.shape, dt),
        *c.act("ddelta", ddelta, u.shape, dt), *c.act("dz", dz, u.shape, dt, True),
        *c.act("dB", dB, B.shape, dt, inner=2), *c.act("dC", dC, B.shape, dt, inner=2),
        *c.grad("dA", dA, (D, N), S), *c.grad("dskip", dskip, (D,), S, True),
        *c.grad("ddelta_bias", ddelta_bias, (D,), S, True),
        *c.states("dstate_out", dstate_out, (R, D, N)),
        *c.states("dstate_in", dstate_in, (R, D, N)))
    need = _call("zo_scan_backward_workspace")(a)
    c.run("zo_scan_backward", a, g, stream=stream, workspace=(workspace, need))


# ---- norms around a block -----------------------------------------------------------

def _norm_args(c, x, x_out, n_out, o, gate, w_post, scale, w_pre, eps, gate_first, like):
    if x.dim() != 2:
        c.fail("x", "must be [rows, channels]")
    dt = like.dtype if like is not None else x.dtype
    R, D = x.shape
    S = _sets((w_post, 1), (scale, 1), (w_pre, 1))
    args = (
        R, D, S, c.code(like if like is not None else x), c.code(x),
        ZO_NORM_GATE_FIRST if gate_first else 0, eps, *c.act("x", x, x.shape, x.dtype),
        *c.act("x_out", x_out, x.shape, x.dtype, True), *c.act("o", o, x.shape, dt, True),
        *c.act("gate", gate, x.shape, dt, True), *c.act("n_out", n_out, x.shape, dt, True),
        *c.param("w_post", w_post, (D,), S, True), *c.param("scale", scale, (D,), S, True),
        *c.param("w_pre", w_pre, (D,), S, True))
    return S, c.pack(NormArgs, args)


def zo_block_norm(x, x_out=None, n_out=None, o=None, gate=None, w_post=None, scale=None,
                  w_pre=None, eps=1e-6, gate_first=False, stream=None):
    """The join of two blocks over rows [rows, channels]:

    p = rms(o) w_post silu(gate) (gate_first: rms(o silu(gate)) w_post), x_out = x + scale p,
    n_out = rms(x_out) w_pre.  Without o only the norm of x.  x may be float32 while the others
    are narrower; x_out may be x."""
    c = _Call("zo_block_norm", x)
    _, a = _norm_args(c, x, x_out, n_out, o, gate, w_post, scale, w_pre, eps, gate_first,
                      o if o is not None else n_out)
    c.run("zo_block_norm", a, stream=stream)


def zo_block_norm_backward(x_out, dn=None, dx_out=None, dx=None, do=None, dgate=None, dw_post=None,
                           dscale=None, dw_pre=None, o=None, gate=None, w_post=None, scale=None,
                           w_pre=None, eps=1e-6, gate_first=False, workspace=None, stream=None):
    """Gradients of zo_block_norm from dn (of n_out) and dx_out (of x_out), at least one of them.

    x_out as zo_block_norm wrote it (x itself where there is no o).  Each gradient is required
    with what it belongs to; dx may be dx_out."""
    c = _Call("zo_block_norm_backward", x_out)
    S, a = _norm_args(c, x_out, x_out, None, o, gate, w_post, scale, w_pre, eps, gate_first,
                      o if o is not None else dn)
    xt, D = x_out.dtype, (x_out.shape[1],)
    dt = (o if o is not None else dn if dn is not None else x_out).dtype
    shape = x_out.shape
    g = _PACK[NormGrads](
        *c.act("dn", dn, shape, dt, True), *c.act("dx_out", dx_out, shape, xt, True),
        *c.act("dx", dx, shape, xt), *c.act("do", do, shape, dt, True),
        *c.act("dgate", dgate, shape, dt, True), *c.grad("dw_post", dw_post, D, S, True),
        *c.grad("dscale", dscale, D, S, True), *c.grad("dw_pre", dw_pre, D, S, True))
    need = _call("zo_block_norm_backward_workspace")(a)
    c.run("zo_block_norm_backward", a, g, stream=stream, workspace=(workspace, need))
