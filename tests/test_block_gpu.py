"""The state-space block's operators on the GPU against the 64-bit references.

Tolerances.  An output of type t is the fp32 result rounded once: half a step,
eps(t) / 2 relative.  The fp32 result is a sum of terms; `size` of the reference is
the sum of the terms' absolute values, and every operation on the way to a term
is off by at most u = 2^-24 relative (exp, log1p and the sigmoid's quotient by a
few u, counted as such below), so the result is off by at most u * size * (the
number of operations on the longest way)."""
import pytest
import torch

import zero_order_recurrent_b200 as zo
from tests import block_reference as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from zero_order_recurrent_b200 import build
    build.build()
    zo.load_library()


def near(got, want, size, ops, what=""):
    """|got - want| <= half a step of got's type + ops * u * size, everywhere."""
    tiny = torch.finfo(got.dtype).tiny  # below it a step is a fixed one
    tol = torch.finfo(got.dtype).eps / 2 * (want.abs() + ops * U * size) + ops * U * size + tiny
    off = (got.double() - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.numel(), float((off / tol).max()))


class Inputs:
    """Seeded tensors; `pad` of them lie in larger buffers of NaN with odd strides."""

    def __init__(self, seed, pad=False):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        self.pad = pad

    def normal(self, *shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=self.g, device="cuda") * scale).to(dtype)

    def act(self, *shape, **kw):
        return self.place(self.normal(*shape, **kw))

    def place(self, v):
        """v, or a copy of it inside a larger buffer: other row and step strides, an odd offset."""
        if not self.pad:
            return v
        big = torch.full((v.shape[0], *(s + 1 for s in v.shape[1:-1]), v.shape[-1] + 3), float("nan"),
                         device="cuda", dtype=v.dtype)
        view = big[(slice(None),) + tuple(slice(0, s) for s in v.shape[1:-1]) + (slice(1, v.shape[-1] + 1),)]
        view.copy_(v)
        return view

    def out(self, *shape, dtype=torch.float32):
        return self.place(torch.full(shape, float("nan"), device="cuda", dtype=dtype))


def lengths_of(kind, R, T, g):
    if kind is None:
        return None
    n = torch.randint(0, T + 1, (R,), generator=g, device="cuda", dtype=torch.int32)
    n[0] = 0
    n[-1] = T
    return n


def poison(t, lengths):
    """NaN and infinity from each row's length on."""
    if lengths is not None:
        for r, n in enumerate(lengths.tolist()):
            t[r, n:] = float("nan") if r % 2 else float("inf")
    return t


def untouched(view):
    """Everything of view's buffer outside view is still NaN."""
    big = view._base
    if big is None:
        return
    mask = torch.ones_like(big, dtype=torch.bool)
    mask[(slice(None),) + tuple(slice(0, s) for s in view.shape[1:-1]) + (slice(1, view.shape[-1] + 1),)] = False
    assert torch.isnan(big[mask]).all()


# ---- convolution --------------------------------------------------------------------

CONV = [  # R, T, D, K, S, dtype, ragged, state, pad, act
    (1, 1, 1, 1, 1, "f32", None, False, False, True),
    (2, 3, 7, 4, 1, "bf16", None, True, False, True),
    (6, 17, 64, 4, 3, "bf16", True, True, False, True),
    (4, 100, 40, 2, 2, "f16", True, True, True, True),
    (3, 65, 136, 3, 1, "f32", True, False, False, False),
    (2, 33, 24, 8, 1, "bf16", True, True, False, True),
    (4, 2, 264, 5, 4, "f16", True, True, False, True),
    (1, 700, 520, 4, 1, "bf16", None, False, False, True),
    (2, 31, 33, 6, 2, "f32", True, True, True, True),
    (3, 5, 8, 7, 1, "f16", True, True, False, False),
    (2, 3000, 24, 4, 1, "bf16", True, True, False, True),
    (3, 40, 30, 4, 3, "bf16", True, True, False, True),
]


@pytest.mark.parametrize("R,T,D,K,S,dtype,ragged,state,pad,act", CONV)
def test_conv(R, T, D, K, S, dtype, ragged, state, pad, act):
    i, dt = Inputs(R * T + D, pad), DT[dtype]
    n = lengths_of(ragged, R, T, i.g)
    x = poison(i.act(R, T, D, dtype=dt), n)
    w, b = i.normal(S, K, D, scale=0.5), i.normal(S, D)
    st = i.act(R, K - 1, D, dtype=dt) if state and K > 1 else None
    out, so = i.out(R, T, D, dtype=dt), i.out(R, K - 1, D, dtype=dt)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    zo.zo_conv(x, w, out, bias=b, silu=act, lengths=n, state_in=st, state_out=so, status=status)
    want, last, _, _ = ref.conv(x, w, b, act, n, st)
    size = ref.conv(x, w, b, act, n, st, size=True)[0]
    near(out, want, size, K + 8, "out")
    assert torch.equal(so.double(), last)
    assert int(status) == 0
    if pad:
        untouched(out)
    if st is not None:  # the window moved in place
        zo.zo_conv(x, w, out, bias=b, silu=act, lengths=n, state_in=st, state_out=st)
        assert torch.equal(st.double(), last)


@pytest.mark.parametrize("R,T,D,K,S,dtype,ragged,state,pad,act", CONV)
def test_conv_backward(R, T, D, K, S, dtype, ragged, state, pad, act):
    i, dt = Inputs(R * T + D + 1, pad), DT[dtype]
    n = lengths_of(ragged, R, T, i.g)
    x, dout = (poison(i.act(R, T, D, dtype=dt), n) for _ in range(2))
    w, b = i.normal(S, K, D, scale=0.5), i.normal(S, D)
    win = (R, K - 1, D)
    st, dso = (i.act(*win, dtype=dt) if state and K > 1 else None for _ in range(2))
    dsi = i.out(*win, dtype=dt) if st is not None else None
    dx = i.out(R, T, D, dtype=dt)
    dw, db = (torch.full(s, float("nan"), device="cuda") for s in ((S, K, D), (S, D)))
    zo.zo_conv_backward(x, w, dout, dx, dw, bias=b, dbias=db, silu=act, lengths=n, state_in=st,
                        dstate_out=dso, dstate_in=dsi)
    args = (x, w, dout, b, act, n, st, dso)
    wants, sizes = ref.conv_backward(*args), ref.conv_backward(*args, size=True)
    ops = 2 * K + 16
    near(dx, wants[0], sizes[0], ops, "dx")
    near(dw, wants[1], sizes[1], ops + R * T // S, "dweight")
    near(db, wants[2], sizes[2], ops + R * T // S, "dbias")
    if dsi is not None:
        near(dsi, wants[3], sizes[3], ops, "dstate_in")
    if pad:
        untouched(dx)


@pytest.mark.parametrize("K,dtype,D", [(1, "bf16", 8), (2, "f32", 5), (4, "bf16", 72), (8, "f16", 33)])
def test_conv_steps_equal_the_prompt(K, dtype, D):
    R, T, dt = 3, 12, DT[dtype]
    i = Inputs(K, False)
    x, w, b = i.act(R, T, D, dtype=dt), i.normal(K, D), i.normal(D)
    out, st = torch.empty_like(x), torch.zeros(R, K - 1, D, dtype=dt, device="cuda")
    zo.zo_conv(x, w, out, bias=b)
    for t in range(T):
        y = torch.empty(R, D, dtype=dt, device="cuda")
        zo.zo_conv_step(x[:, t], w, st, y, bias=b)
        assert torch.equal(y, out[:, t])


# ---- scan ---------------------------------------------------------------------------

SCAN = [  # R, T, D, G, N, S, dtype, ragged, state, gate, softplus, pad
    (1, 1, 1, 1, 1, 1, "f32", None, False, False, False, False),
    (2, 5, 40, 1, 16, 1, "bf16", None, True, True, True, False),
    (4, 33, 64, 2, 16, 2, "f32", True, True, True, True, False),
    (3, 50, 24, 4, 7, 1, "f16", True, True, False, True, True),
    (6, 16, 17, 1, 4, 3, "f32", True, False, True, True, False),
    (2, 100, 36, 1, 24, 1, "bf16", True, True, True, True, False),
    (2, 31, 10, 1, 64, 1, "f32", None, True, True, True, True),
    (1, 40, 6, 2, 128, 1, "f32", True, True, True, False, False),
    (1, 300, 130, 1, 16, 1, "bf16", None, True, True, True, False),
    (2, 17, 33, 3, 2, 2, "f32", True, True, False, False, False),
    (1, 65, 8, 8, 33, 1, "f16", None, False, True, True, False),
    (5, 2, 96, 1, 16, 5, "bf16", True, True, True, True, True),
    (1, 2500, 16, 1, 16, 1, "f32", None, True, True, True, False),
    (230, 1100, 8, 1, 16, 2, "f32", True, False, True, True, False),
    (650, 40, 8, 1, 16, 2, "f32", True, True, False, True, False),
    (6000, 5, 8, 1, 16, 3, "bf16", True, True, True, True, False),
    (2600, 40, 40, 1, 8, 1, "f16", True, False, True, True, False),
]


def scan_inputs(R, T, D, G, N, S, dtype, ragged, state, gate, softplus, pad, seed=0):
    i, dt = Inputs(seed + R * T + D + N, pad), DT[dtype]
    n = lengths_of(ragged, R, T, i.g)
    u, dl, z = (poison(i.act(R, T, D, dtype=dt), n) for _ in range(3))
    dl.copy_(dl if softplus else dl.abs())
    if pad:
        B, C = (i.act(R, T, G * N, dtype=dt) for _ in range(2))
        B, C = (t.unflatten(2, (G, N)) for t in (poison(B, n), poison(C, n)))
    else:
        B, C = (poison(i.act(R, T, G, N, dtype=dt), n) for _ in range(2))
    A = -torch.rand(S, D, N, generator=i.g, device="cuda") * 2
    skip, bias = i.normal(S, D), i.normal(S, D)
    if not softplus:
        bias = bias.abs()
    st = i.normal(R, D, N) if state else None
    return i, n, u, dl, A, B, C, dict(skip=skip, z=z if gate else None), bias, st


# operations on a term's way: per step the exponent's argument (|d A| u by the softplus's 6 u and
# the product), the exponential's 4 u, a multiplication and an addition, for as many steps as there
# are; then the sums over states, channels, rows
def scan_ops(T, N, dl, A, bias, softplus, extra=0):
    _, d = ref.steps(torch.nan_to_num(dl.double(), 0, 0, 0), bias, softplus)
    da = float((d.amax(1) * ref.each(A, dl.shape[0]).abs().amax(-1)).max())
    return T * (8 + 8 * da) + N + 24 + extra


@pytest.mark.parametrize("R,T,D,G,N,S,dtype,ragged,state,gate,softplus,pad", SCAN)
def test_scan(R, T, D, G, N, S, dtype, ragged, state, gate, softplus, pad):
    i, n, u, dl, A, B, C, kw, bias, st = scan_inputs(R, T, D, G, N, S, dtype, ragged, state, gate, softplus, pad)
    out, so = i.out(R, T, D, dtype=u.dtype), torch.full((R, D, N), float("nan"), device="cuda")
    if pad:
        so = torch.full((R, 2, D, N), float("nan"), device="cuda")[:, 0]
    kept = torch.full(zo.zo_scan_checkpoint_shape(u.shape, N), float("nan"), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    zo.zo_scan(u, dl, A, B, C, out, delta_bias=bias, softplus=softplus, lengths=n, state_in=st,
               state_out=so, checkpoints=kept, status=status, **kw)
    args = (u, dl, A, B, C, kw["skip"], kw["z"], bias, softplus, n, st)
    (want, last, hs, _), (size, slast, shs, _) = ref.scan(*args), ref.scan(*args, size=True)
    ops = scan_ops(T, N, dl, A, bias, softplus)
    near(out, want, size, ops, "out")
    near(so, last, slast, ops, "state_out")
    near(kept, hs[:, :-1][:, ::zo.ZO_SCAN_CHUNK], shs[:, :-1][:, ::zo.ZO_SCAN_CHUNK], ops, "checkpoints")
    assert int(status) == 0
    again = torch.empty_like(out)
    zo.zo_scan(u, dl, A, B, C, again, delta_bias=bias, softplus=softplus, lengths=n, state_in=st, **kw)
    near(again, want, size, ops, "without checkpoints")
    if pad:
        untouched(out)
    if st is not None:  # the state moved in place
        zo.zo_scan(u, dl, A, B, C, again, delta_bias=bias, softplus=softplus, lengths=n, state_in=st,
                   state_out=st, **kw)
        near(st, last, slast, ops, "state in place")


@pytest.mark.parametrize("R,T,D,G,N,S,dtype,ragged,state,gate,softplus,pad", SCAN)
def test_scan_backward(R, T, D, G, N, S, dtype, ragged, state, gate, softplus, pad):
    i, n, u, dl, A, B, C, kw, bias, st = scan_inputs(R, T, D, G, N, S, dtype, ragged, state, gate, softplus, pad, 1)
    dt = u.dtype
    out, dout = torch.empty(R, T, D, dtype=dt, device="cuda"), poison(i.act(R, T, D, dtype=dt), n)
    kept = torch.empty(zo.zo_scan_checkpoint_shape(u.shape, N), device="cuda")
    zo.zo_scan(u, dl, A, B, C, out, delta_bias=bias, softplus=softplus, lengths=n, state_in=st,
               checkpoints=kept, **kw)
    du, dd = i.out(R, T, D, dtype=dt), i.out(R, T, D, dtype=dt)
    dz = i.out(R, T, D, dtype=dt) if gate else None
    dB, dC = (torch.full((R, T, G, N), float("nan"), dtype=dt, device="cuda") for _ in range(2))
    dA, dskip, dbias = (torch.full(s, float("nan"), device="cuda") for s in ((S, D, N), (S, D), (S, D)))
    dso = i.normal(R, D, N) if state else None
    dsi = torch.full((R, D, N), float("nan"), device="cuda") if state else None
    zo.zo_scan_backward(u, dl, A, B, C, dout, kept, du, dd, dA, dB, dC, dskip=dskip, dz=dz,
                        delta_bias=bias, ddelta_bias=dbias, softplus=softplus, lengths=n,
                        dstate_out=dso, dstate_in=dsi, **kw)
    args = (u, dl, A, B, C, dout, kw["skip"], kw["z"], bias, softplus, n, st, dso)
    want, size = ref.scan_backward(*args), ref.scan_backward(*args, size=True)
    # both directions of time, and the states once more
    ops = 2 * scan_ops(T, N, dl, A, bias, softplus) + 16
    for name, got, extra in (("du", du, 0), ("ddelta", dd, 0), ("dz", dz, 0), ("dB", dB, D // G), ("dC", dC, D // G),
                             ("dA", dA, T * R // S), ("dskip", dskip, T * R // S), ("ddelta_bias", dbias, T * R // S),
                             ("dstate_in", dsi, 0)):
        if got is not None:
            near(got, want[name], size[name], ops + extra, name)
    if pad:
        untouched(du)
        untouched(dd)


@pytest.mark.parametrize("D,G,N,dtype,gate", [(40, 1, 16, "bf16", True), (6, 2, 3, "f32", False), (20, 1, 64, "f16", True)])
def test_scan_steps_equal_the_prompt(D, G, N, dtype, gate):
    R, T = 3, 9
    i, _, u, dl, A, B, C, kw, bias, st = scan_inputs(R, T, D, G, N, 1, dtype, None, True, gate, True, False, 2)
    out, so, now = torch.empty_like(u), torch.empty_like(st), st.clone()
    zo.zo_scan(u, dl, A, B, C, out, delta_bias=bias, state_in=st, state_out=so, **kw)
    args = (u, dl, A, B, C, kw["skip"], kw["z"], bias, True, None, st)
    (want, last, _, _), (size, slast, _, _) = ref.scan(*args), ref.scan(*args, size=True)
    ops = scan_ops(T, N, dl, A, bias, True)
    y = torch.empty_like(u)
    z = kw.pop("z")
    for t in range(T):
        zo.zo_scan_step(u[:, t], dl[:, t], A, B[:, t], C[:, t], now, y[:, t], delta_bias=bias,
                        z=None if z is None else z[:, t], **kw)
    near(y, want, size, ops, "steps")
    near(now, last, slast, ops, "state")
    near(so, last, slast, ops, "prompt's state")


@pytest.mark.parametrize("A", [-3.4e38, -1e30, -1e-30, 0.0, 0.3])
def test_scan_extreme_decays(A):
    """Decays of 0 and 1 and above, steps of length 0 between them, and their gradients."""
    R, T, D, N = 2, 40, 8, 4
    i = Inputs(7, False)
    u, B, C, dout = i.normal(R, T, D), i.normal(R, T, 1, N), i.normal(R, T, 1, N), i.normal(R, T, D)
    dl = i.normal(R, T, D).abs() * (torch.rand(R, T, D, generator=i.g, device="cuda") < 0.7)
    a, st = torch.full((1, D, N), A, device="cuda"), i.normal(R, D, N)
    out, so = torch.empty_like(u), torch.empty_like(st)
    kept = torch.empty(zo.zo_scan_checkpoint_shape(u.shape, N), device="cuda")
    zo.zo_scan(u, dl, a, B, C, out, softplus=False, state_in=st, state_out=so, checkpoints=kept)
    args = (u, dl, a, B, C, None, None, None, False, None, st)
    (want, last, _, _), (size, slast, _, _) = ref.scan(*args), ref.scan(*args, size=True)
    # |d A| matters only where the decay is not 0: up to 104, from where fp32 has none
    ops = T * (8 + 8 * min(104.0, float(dl.max()) * abs(A))) + 64
    near(out, want, size, ops, "out")
    near(so, last, slast, ops, "state")
    g = {k: torch.empty_like(t) for k, t in {"du": u, "ddelta": dl, "dA": a, "dB": B, "dC": C}.items()}
    zo.zo_scan_backward(u, dl, a, B, C, dout, kept, g["du"], g["ddelta"], g["dA"], g["dB"], g["dC"], softplus=False)
    # rates count up to the largest fp32 over log2(e) (include/zo_block.h)
    args = (u, dl, a.double().clamp(min=-torch.finfo(torch.float32).max / 1.4426950408889634), B, C,
            dout, None, None, None, False, None, st)
    want, size = ref.scan_backward(*args), ref.scan_backward(*args, size=True)
    for k in g:
        # at steps of length 0, ddelta has terms g A h, which are summed as g (A log2(e)) h: where
        # those add up to more than the largest fp32, 3.4e38, each or a partial sum can be
        # infinite though the sum is not, and fp32 has no answer
        fits = size[k] * 1.4426950408889634 < torch.finfo(torch.float32).max
        near(g[k][fits], want[k][fits], size[k][fits], 2 * ops + T * R, k)
        assert fits.all() or (k == "ddelta" and A < -1e37)


@pytest.mark.parametrize("small", [False, True])
def test_scan_growth_beyond_fp32_over_a_part(small):
    """Growing states: one row's time is divided in parts, and e^128 over 32 steps is beyond fp32
    though what it multiplies, 0 (small: 1e-30), leaves the state in range."""
    T, D, N = 128, 8, 4
    i = Inputs(9, False)
    u, B, C, dout = i.normal(1, T, D), i.normal(1, T, 1, N), i.normal(1, T, 1, N), i.normal(1, T, D)
    a, dl = torch.full((1, D, N), 4.0, device="cuda"), torch.ones(1, T, D, device="cuda")
    # T * (a step's operations, and |d A| = 4 in units of the exponent's error) as above
    ops = T * (8 + 8 * 4) + 64

    def forward(u, dl, st):
        out, so = torch.empty_like(u), torch.empty(1, D, N, device="cuda")
        kept = torch.empty(zo.zo_scan_checkpoint_shape(u.shape, N), device="cuda")
        zo.zo_scan(u, dl, a, B, C, out, softplus=False, state_in=st, state_out=so, checkpoints=kept)
        args = (u, dl, a, B, C, None, None, None, False, None, st)
        (want, last, _, _), (size, slast, _, _) = ref.scan(*args), ref.scan(*args, size=True)
        near(out, want, size, ops, "out")
        near(so, last, slast, ops, "state")
        return kept

    v, d = u.clone(), dl.clone()
    if small:
        v[:], d[:, 32:] = 0, 0
        forward(v, d, 1e-30 * i.normal(1, D, N))
    else:
        v[:, :-8] = 0
        forward(v, d, None)

    v, d, ds = u.clone(), dl.clone(), None
    if small:
        v[:, -32:], d[:, :-32], ds = 0, 0, 1e-30 * i.normal(1, D, N)
        dout[:] = 0
    else:
        v[:], dout[:, 8:] = 0, 0
    kept = forward(v, d, None)
    g = {k: torch.empty_like(t) for k, t in {"du": v, "ddelta": d, "dA": a, "dB": B, "dC": C}.items()}
    zo.zo_scan_backward(v, d, a, B, C, dout, kept, g["du"], g["ddelta"], g["dA"], g["dB"], g["dC"],
                        softplus=False, dstate_out=ds)
    args = (v, d, a, B, C, dout, None, None, None, False, None, None, ds)
    want, size = ref.scan_backward(*args), ref.scan_backward(*args, size=True)
    for k in g:
        near(g[k], want[k], size[k], 2 * ops + T, k)


def test_scan_gradient_against_differences():
    """The kernel's gradients against central differences of the kernel's own forward."""
    R, T, D, N = 2, 12, 8, 4
    i, n, u, dl, A, B, C, kw, bias, st = scan_inputs(R, T, D, 1, N, 1, "f32", True, True, True, True, False, 5)
    dout = torch.nan_to_num(i.normal(R, T, D))
    tensors = {"du": u, "ddelta": dl, "dA": A, "dB": B, "dC": C, "dz": kw["z"], "dskip": kw["skip"], "ddelta_bias": bias}
    out = torch.empty_like(u)
    kept = torch.empty(zo.zo_scan_checkpoint_shape(u.shape, N), device="cuda")
    call = dict(delta_bias=bias, lengths=n, state_in=st, **kw)

    def f():
        zo.zo_scan(u, dl, A, B, C, out, checkpoints=kept, **call)
        return float((out.double() * dout.double()).sum())

    f()
    g = {k: torch.empty_like(t) for k, t in tensors.items()}
    call.pop("state_in")
    zo.zo_scan_backward(u, dl, A, B, C, dout, kept, g["du"], g["ddelta"], g["dA"], g["dB"], g["dC"],
                        dskip=g["dskip"], dz=g["dz"], ddelta_bias=g["ddelta_bias"], **call)
    call["state_in"] = st
    h = 2.0 ** -7
    scale = float(dout.double().abs().sum() * out.double().abs().max())
    for name, t in tensors.items():
        v = torch.where(torch.isfinite(t), torch.randn(t.shape, generator=i.g, device="cuda"), 0.0)
        v = v / v.norm()
        keep, vals = t.clone(), []
        for s in (h, -h):
            t.copy_(keep + s * v)
            vals.append(f())
        t.copy_(keep)
        want = (vals[0] - vals[1]) / (2 * h)
        got = float((g[name].double() * v.double()).sum())
        # the quotient: fp32 forwards, 300 u of the loss's size over 2 h; third derivatives, of the
        # order of the loss's size, times h^2 / 6
        assert abs(got - want) <= scale * (300 * U / (2 * h) + h * h), (name, got, want)


# ---- norms ----------------------------------------------------------------------------

NORM = [  # R, D, S, dtype, residual, without, gate_first, pad
    (1, 1, 1, "f32", "f32", (), False, False),
    (5, 64, 1, "bf16", "f32", (), False, False),
    (6, 264, 3, "bf16", "bf16", (), True, False),
    (4, 1000, 2, "f16", "f32", ("gate",), False, False),
    (3, 333, 1, "f16", "f16", ("scale",), False, True),
    (2, 2048, 1, "bf16", "f32", ("w_post",), False, False),
    (3, 4097, 1, "f32", "f32", (), True, False),
    (7, 8192, 1, "bf16", "f32", (), False, False),
    (2, 16384, 1, "bf16", "bf16", (), False, False),
    (3, 9001, 3, "bf16", "f32", ("w_post",), True, False),
    (4, 72, 2, "f32", "f32", ("o", "gate", "w_post", "scale"), False, False),
    (3, 520, 1, "bf16", "f32", ("w_pre",), False, True),
    (600, 40, 2, "bf16", "f32", (), False, False),
    (1300, 2056, 1, "f16", "f32", (), False, False),
]


def norm_inputs(R, D, S, dtype, residual, without, pad, seed=0):
    i = Inputs(R + D + seed, pad)
    dt, xt = DT[dtype], DT[residual]
    p = {"o": i.act(R, D, dtype=dt, scale=0.5), "gate": i.act(R, D, dtype=dt), "w_post": i.normal(S, D),
         "scale": i.normal(S, D), "w_pre": i.normal(S, D)}
    for k in without:
        p.pop(k)
    return i, dt, xt, i.act(R, D, dtype=xt), p


def rows_size(v):
    return v.abs() + v.pow(2).mean(1, keepdim=True).sqrt()


@pytest.mark.parametrize("R,D,S,dtype,residual,without,gate_first,pad", NORM)
def test_norm(R, D, S, dtype, residual, without, gate_first, pad):
    i, dt, xt, x, p = norm_inputs(R, D, S, dtype, residual, without, pad)
    xo = i.out(R, D, dtype=xt)
    no = i.out(R, D, dtype=dt) if "w_pre" in p else None
    zo.zo_block_norm(x, x_out=xo, n_out=no, eps=1e-5, gate_first=gate_first, **p)
    want, wn = ref.norm(x, eps=1e-5, gate_first=gate_first, **p)
    # the norms' sums of D squares are off by D u of themselves, their roots by half that
    ops = D / 2 + 24
    add = (want - x.double()).abs()
    near(xo, want, x.double().abs() + add, ops, "x_out")
    if no is not None:
        near(no, wn, wn.abs() + rows_size(x.double().abs() + add) / rows_size(want) * ref.each(p["w_pre"], R).abs() * 4,
             2 * ops, "n_out")
    if pad:
        untouched(xo)
    if "w_pre" in p:  # without x_out, and in place
        again = torch.empty(R, D, dtype=dt, device="cuda")
        zo.zo_block_norm(x, n_out=again, eps=1e-5, gate_first=gate_first, **p)
        assert torch.equal(again, no)
    zo.zo_block_norm(x, x_out=x, n_out=no, eps=1e-5, gate_first=gate_first, **p)
    assert torch.equal(x, xo)


@pytest.mark.parametrize("R,D,S,dtype,residual,without,gate_first,pad", NORM)
def test_norm_backward(R, D, S, dtype, residual, without, gate_first, pad):
    i, dt, xt, y, p = norm_inputs(R, D, S, dtype, residual, without, pad, 1)
    dn = i.act(R, D, dtype=dt) if "w_pre" in p else None
    dxo = None if R == 5 else i.act(R, D, dtype=xt)
    got = {"dx": i.out(R, D, dtype=xt)}
    got |= {"d" + k: i.out(R, D, dtype=dt) for k in ("o", "gate") if k in p}
    got |= {"d" + k: torch.full((S, D), float("nan"), device="cuda") for k in ("w_post", "scale", "w_pre") if k in p}
    zo.zo_block_norm_backward(y, dn=dn, dx_out=dxo, eps=1e-5, gate_first=gate_first, **got, **p)
    want = ref.norm_backward(y, dn, dxo, eps=1e-5, gate_first=gate_first, **p)
    # Sizes: |G| <= |dx_out| + rn (|e| + |y rn| mean |e y rn|), e = dn w_pre, and what follows from it
    # linearly; each of the two norms' sums adds D / 2 + 1 operations
    ops = D + 64
    f = lambda v: v.double().abs()  # noqa: E731
    G = torch.zeros(R, D, dtype=torch.float64, device="cuda") if dxo is None else f(dxo)
    if dn is not None:
        rn = 1 / torch.sqrt((f(y) ** 2).mean(1, keepdim=True) + 1e-5)
        e, yh = f(dn) * f(ref.each(p["w_pre"], R)), f(y) * rn
        G = G + rn * (e + yh * (e * yh).mean(1, keepdim=True))
        near(got["dw_pre"], want["dw_pre"], ref.by_set(f(dn) * yh, S), ops + R // S, "dw_pre")
    near(got["dx"], want["dx"], G, ops, "dx")
    if "o" in p:
        o = f(p["o"])
        z = p["gate"].double() if "gate" in p else None
        act = torch.ones_like(o) if z is None else f(ref.silu(z))
        one = torch.ones_like(o)
        v, after = (o * act, one) if gate_first else (o, act)
        wp = f(ref.each(p["w_post"], R)) if "w_post" in p else one
        sc = f(ref.each(p["scale"], R)) if "scale" in p else one
        vh = v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-5) if "w_post" in p else v
        r = 1 / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-5) if "w_post" in p else 1.0
        dvh = G * sc * after * wp
        dv = r * (dvh + vh * (dvh * vh).mean(1, keepdim=True)) if "w_post" in p else dvh
        near(got["do"], want["do"], dv * act if gate_first else dv, 2 * ops, "do")
        if z is not None:
            near(got["dgate"], want["dgate"], 1.1 * (dv * o if gate_first else G * sc * vh * wp), 2 * ops, "dgate")
        if "w_post" in p:
            near(got["dw_post"], want["dw_post"], ref.by_set(G * sc * after * vh, S), 2 * ops + R // S, "dw_post")
        if "scale" in p:
            near(got["dscale"], want["dscale"], ref.by_set(G * vh * wp * after, S), 2 * ops + R // S, "dscale")
    if pad:
        untouched(got["dx"])
    if dxo is not None:  # the residual's gradient in place
        more = {k: torch.empty_like(v) for k, v in got.items() if k != "dx"}
        zo.zo_block_norm_backward(y, dn=dn, dx_out=dxo, dx=dxo, eps=1e-5, gate_first=gate_first, **more, **p)
        assert torch.equal(dxo, got["dx"])
