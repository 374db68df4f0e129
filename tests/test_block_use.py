"""The state-space block's operators as they are used: together, with probe losses, on
streams and in CUDA graphs; and what they refuse."""
import ctypes

import pytest
import torch

import zero_order_recurrent_b200 as zo
from tests import block_reference as ref
from zero_order_recurrent_b200 import block

gpu = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def library():
    from zero_order_recurrent_b200 import build
    build.build()
    zo.load_library()


# ---- refusals, without a device -----------------------------------------------------

P = 1 << 20  # an address that is only looked at


def conv_args(**kw):
    t = block._Tensor(P, 64, 8)
    a = block.ConvArgs(2, 4, 8, 4, 1, zo.ZO_DTYPE_FP32, 1, t, block._Tensor(2 * P, 64, 8), block._F32(P, 0))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def scan_args(**kw):
    t, bc = block._Tensor(P, 64, 8), block._Tensor(P, 64, 16)
    a = block.ScanArgs(2, 4, 8, 1, 16, 1, zo.ZO_DTYPE_FP32, 1, t, t, block._Tensor(2 * P, 64, 8), block._Tensor(),
                       bc, bc, block._F32(P, 0))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def norm_args(**kw):
    t = block._Tensor(P, 8, 0)
    a = block.NormArgs(4, 8, 1, zo.ZO_DTYPE_FP32, zo.ZO_DTYPE_FP32, 0, 1e-5, t, block._Tensor(2 * P, 8, 0))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


BAD_SIZES = [dict(rows=0), dict(rows=-1), dict(channels=0), dict(channels=2 ** 30 + 2), dict(sets=0), dict(sets=3), dict(dtype=7), dict(flags=8)]
T0, F0 = block._Tensor(), block._F32()


@pytest.mark.parametrize("kw", BAD_SIZES + [
    dict(seq=0), dict(seq=2 ** 30 + 1), dict(taps=0), dict(x=T0), dict(out=T0), dict(weight=F0), dict(x=block._Tensor(P + 2, 64, 8)),
    dict(out=block._Tensor(P, 64, 8)), dict(out=block._Tensor(2 * P, 64, 7)), dict(out=block._Tensor(2 * P, 16, 8)),
    dict(lengths=P + 1), dict(state_in=block._Tensor(P + 1, 24, 8)), dict(state_out=block._Tensor(3 * P, 16, 8)),
    dict(state_in=block._Tensor(3 * P, 24, 8), state_out=block._Tensor(3 * P, 32, 8))])
def test_conv_refuses(kw):
    lib = zo.load_library()
    assert lib.zo_conv(conv_args(**kw), None) == zo.ZO_ERR_INVALID_ARG


def test_conv_refuses_more():
    lib = zo.load_library()
    assert lib.zo_conv(None, None) == zo.ZO_ERR_INVALID_ARG
    assert lib.zo_conv(conv_args(taps=9), None) == zo.ZO_ERR_UNSUPPORTED
    assert lib.zo_conv_step(conv_args(), None) == zo.ZO_ERR_INVALID_ARG            # seq != 1
    assert lib.zo_conv_step(conv_args(seq=1), None) == zo.ZO_ERR_INVALID_ARG       # no window
    assert lib.zo_conv_backward_workspace(conv_args(taps=9)) == -1
    a = conv_args()
    need = lib.zo_conv_backward_workspace(a)
    assert need > 0
    t = block._Tensor(3 * P, 64, 8)
    good = (t, block._Tensor(4 * P, 64, 8), block._F32(5 * P, 0))
    for g, ws, n in ((block.ConvGrads(), P, need), (block.ConvGrads(*good), None, need),
                     (block.ConvGrads(*good), P, need - 1), (block.ConvGrads(*good), P + 4, need),
                     (block.ConvGrads(t, t, block._F32(5 * P, 0)), P, need),
                     (block.ConvGrads(t, block._Tensor(P, 64, 8), block._F32(5 * P, 0)), P, need)):
        assert lib.zo_conv_backward(a, g, ws, n, None) == zo.ZO_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", BAD_SIZES + [
    dict(seq=0), dict(seq=2 ** 30 + 1), dict(groups=0), dict(groups=3), dict(states=0), dict(u=T0), dict(delta=T0), dict(B=T0), dict(C=T0),
    dict(A=F0), dict(out=T0), dict(out=block._Tensor(P, 64, 8)), dict(out=block._Tensor(2 * P, 0, 8)),
    dict(checkpoints=P + 4), dict(state_out=block._F32(3 * P, 64)),
    dict(state_in=block._F32(3 * P, 128), state_out=block._F32(3 * P, 256))])
def test_scan_refuses(kw):
    lib = zo.load_library()
    assert lib.zo_scan(scan_args(**kw), P, 1 << 40, None) == zo.ZO_ERR_INVALID_ARG


def test_scan_refuses_more():
    lib = zo.load_library()
    assert lib.zo_scan(scan_args(states=129), P, 1 << 40, None) == zo.ZO_ERR_UNSUPPORTED
    assert lib.zo_scan_step(scan_args(), None) == zo.ZO_ERR_INVALID_ARG
    assert lib.zo_scan_step(scan_args(seq=1), None) == zo.ZO_ERR_INVALID_ARG
    assert lib.zo_scan_workspace(scan_args(states=129)) == -1
    long = scan_args(rows=1, seq=1 << 16)  # a size that divides time
    if lib.zo_scan_workspace(long):
        assert lib.zo_scan(long, None, 0, None) == zo.ZO_ERR_INVALID_ARG
    a = scan_args(checkpoints=P)
    need = lib.zo_scan_backward_workspace(a)
    t, bc = block._Tensor(3 * P, 64, 8), block._Tensor(3 * P, 64, 16)
    good = dict(dout=t, du=t, ddelta=t, dB=bc, dC=bc, dA=block._F32(P, 0))
    bad = [{k: (T0 if k != "dA" else F0)} for k in good]
    bad += [dict(dz=t), dict(dskip=block._F32(P, 0)), dict(ddelta_bias=block._F32(P, 0)),
            dict(dB=block._Tensor(3 * P, 64, 15)), dict(dstate_in=block._F32(P, 100))]
    for kw in bad:
        g = block.ScanGrads(**{**good, **kw})
        assert lib.zo_scan_backward(a, g, P, need, None) == zo.ZO_ERR_INVALID_ARG, kw
    assert lib.zo_scan_backward(a, block.ScanGrads(**good), P, need - 1, None) == zo.ZO_ERR_INVALID_ARG
    assert lib.zo_scan_backward(scan_args(), block.ScanGrads(**good), P, need, None) == zo.ZO_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", BAD_SIZES + [
    dict(x=T0), dict(x_out=T0), dict(eps=0.0), dict(eps=float("inf")), dict(eps=float("nan")), dict(x_dtype=zo.ZO_DTYPE_BF16),
    dict(gate=block._Tensor(P, 8, 0)), dict(scale=block._F32(P, 0)), dict(w_post=block._F32(P, 0)),
    dict(n_out=block._Tensor(3 * P, 8, 0)), dict(w_pre=block._F32(P, 0)), dict(flags=1, o=block._Tensor(P, 8, 0)),
    dict(x_out=block._Tensor(2 * P, 7, 0)), dict(x_out=block._Tensor(P, 16, 0)),
    dict(n_out=block._Tensor(P, 8, 0), w_pre=block._F32(P, 0))])
def test_norm_refuses(kw):
    lib = zo.load_library()
    assert lib.zo_block_norm(norm_args(**kw), None) == zo.ZO_ERR_INVALID_ARG


def test_norm_refuses_more():
    lib = zo.load_library()
    assert lib.zo_block_norm(norm_args(channels=16385), None) == zo.ZO_ERR_UNSUPPORTED
    a = norm_args(w_pre=block._F32(P, 0))
    need = lib.zo_block_norm_backward_workspace(a)
    t, f = block._Tensor(3 * P, 8, 0), block._F32(P, 0)
    good = dict(dn=t, dx=t, dw_pre=f)
    for kw in (dict(dn=T0), dict(dx=T0), dict(dw_pre=F0), dict(d_o=t), dict(dgate=t), dict(dscale=f), dict(dw_post=f),
               dict(dx=block._Tensor(2 * P, 8, 0)), dict(dx=block._Tensor(3 * P, 4, 0))):
        g = block.NormGrads(**{**good, **kw})
        assert lib.zo_block_norm_backward(a, g, P, need, None) == zo.ZO_ERR_INVALID_ARG, kw
    assert lib.zo_block_norm_backward(a, block.NormGrads(**good), P, need - 1, None) == zo.ZO_ERR_INVALID_ARG


def test_workspaces_of_all_sizes():
    """The plans behind the workspaces, over rows, steps, channels, groups and states: sizes that
    every block arithmetic has to get through, without a device."""
    lib = zo.load_library()
    for rows in (1, 2, 7, 100, 591, 592, 593, 650, 788, 789, 790, 5000, 2 ** 20):
        for seq in (1, 15, 16, 17, 33, 64, 1000, 2 ** 20, 2 ** 30):
            for channels, groups in ((1, 1), (8, 1), (32, 1), (33, 1), (96, 2), (520, 4), (4096, 1), (2 ** 20, 8)):
                if rows * seq * channels > 2 ** 44:
                    continue
                for states in (1, 4, 5, 8, 16, 17, 64, 128):
                    a = scan_args(rows=rows, seq=seq, channels=channels, groups=groups, states=states)
                    n = lib.zo_scan_workspace(a)
                    parts = n // (4 * rows * channels * (states + 1))
                    assert n == parts * 4 * rows * channels * (states + 1) and (parts == 0 or 2 <= parts <= seq)
                    assert lib.zo_scan_backward_workspace(a) > 4 * rows * channels * states
                a = conv_args(rows=rows, seq=seq, channels=channels)
                assert lib.zo_conv_backward_workspace(a) >= 4 * rows * channels * 5
            if channels <= 16384:
                assert lib.zo_block_norm_backward_workspace(norm_args(rows=rows, channels=channels)) > 0


def test_calls_without_a_device_report_it():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    lib = zo.load_library()
    assert lib.zo_conv(conv_args(), None) == zo.ZO_ERR_NO_DEVICE
    assert lib.zo_scan(scan_args(), P, 1 << 40, None) == zo.ZO_ERR_NO_DEVICE
    assert lib.zo_block_norm(norm_args(), None) == zo.ZO_ERR_NO_DEVICE


def test_checkpoint_shape():
    assert zo.zo_scan_checkpoint_shape((2, 1, 8), 4) == (2, 1, 8, 4)
    assert zo.zo_scan_checkpoint_shape((2, 33, 8), 4) == (2, 3, 8, 4)


def test_host_tensors_are_refused():
    x = torch.zeros(2, 3, 8)
    for f in (lambda: zo.zo_conv(x, x, x), lambda: zo.zo_scan(x, x, x, x, x, x), lambda: zo.zo_block_norm(x[0])):
        with pytest.raises(ValueError):
            f()


# ---- refusals of tensors that do not fit together -----------------------------------

@gpu
def test_tensors_are_checked_against_one_another():
    def z(*s, dtype=torch.bfloat16):
        return torch.zeros(*s, dtype=dtype, device="cuda")
    f32 = torch.float32
    x, w = z(4, 6, 16), z(4, 16, dtype=f32)
    good = [x, w, z(4, 6, 16)]
    for at, bad in ((0, z(4, 16)), (1, z(4, 16)), (1, z(4, 15, dtype=f32)), (1, z(3, 4, 16, dtype=f32)),
                    (2, z(4, 6, 16, dtype=f32)), (2, z(4, 6, 17)), (2, z(4, 16, 6).transpose(1, 2)), (2, torch.zeros(4, 6, 16))):
        args = list(good)
        args[at] = bad
        with pytest.raises((ValueError, zo.ZOError)):
            zo.zo_conv(*args)
    for kw in (dict(lengths=z(4, dtype=torch.int64)), dict(lengths=z(3, dtype=torch.int32)), dict(state_in=z(4, 4, 16)),
               dict(bias=z(15, dtype=f32)), dict(bias=z(3, 16, dtype=f32)), dict(status=z(2, dtype=torch.int32))):
        with pytest.raises((ValueError, zo.ZOError)):
            zo.zo_conv(*good, **kw)
    u, A, B = z(4, 6, 16), z(16, 8, dtype=f32), z(4, 6, 2, 8)
    with pytest.raises(ValueError):
        zo.zo_scan(u, u, A, B, z(4, 6, 1, 8), z(4, 6, 16))
    with pytest.raises(ValueError):
        zo.zo_scan(u, u, A, B, B, z(4, 6, 16), state_in=z(4, 16, 8))
    with pytest.raises(ValueError):
        zo.zo_scan(u, u, A, B, B, z(4, 6, 16), checkpoints=z(4, 2, 16, 8, dtype=f32))
    with pytest.raises(zo.ZOError):
        zo.zo_scan(u, u, z(16, 129, dtype=f32), z(4, 6, 1, 129), z(4, 6, 1, 129), z(4, 6, 16))
    with pytest.raises(zo.ZOError):
        zo.zo_scan(u, u, A, z(4, 6, 3, 8), z(4, 6, 3, 8), z(4, 6, 16))  # 3 groups of 16 channels
    with pytest.raises(zo.ZOError):
        zo.zo_block_norm(u[:, 0], n_out=z(4, 16))                       # no w_pre
    with pytest.raises(ValueError):
        zo.zo_block_norm(u[:, 0], x_out=z(4, 16, dtype=f32))


@gpu
def test_launch_failures_are_reported(monkeypatch):
    x, w = torch.ones(2, 3, 8, device="cuda"), torch.ones(4, 8, device="cuda")
    out = torch.full_like(x, 7.0)
    monkeypatch.setenv("ZO_FAULT", "launch")
    with pytest.raises(zo.ZOError) as e:
        zo.zo_conv(x, w, out)
    assert e.value.status == zo.ZO_ERR_CUDA
    monkeypatch.delenv("ZO_FAULT")
    torch.cuda.synchronize()
    assert torch.all(out == 7.0)


@gpu
@pytest.mark.parametrize("bad", [-1, 7, 2 ** 31 - 1, -2 ** 31])
def test_lengths_out_of_range_are_clamped_and_told(bad):
    x, w = torch.randn(2, 6, 8, device="cuda"), torch.randn(4, 8, device="cuda")
    n = torch.tensor([3, bad], dtype=torch.int32, device="cuda")
    ok = torch.tensor([3, 0 if bad < 0 else 6], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    a, b = torch.empty_like(x), torch.empty_like(x)
    zo.zo_conv(x, w, a, lengths=n, status=status)
    zo.zo_conv(x, w, b, lengths=ok)
    assert torch.equal(a, b) and int(status) == zo.ZO_ERR_BOUNDS
    status.zero_()
    A, B = -torch.rand(8, 4, device="cuda"), torch.randn(2, 6, 1, 4, device="cuda")
    zo.zo_scan(x, x, A, B, B, a, lengths=n, status=status)
    zo.zo_scan(x, x, A, B, B, b, lengths=ok)
    assert torch.equal(a, b) and int(status) == zo.ZO_ERR_BOUNDS


# ---- together -----------------------------------------------------------------------

class Block:
    """norm -> in-projection -> convolution -> scan -> out-projection -> norm, with S parameter
    sets for the small parameters; projections by torch."""

    def __init__(self, D, E, N, S, dtype, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def r(*s, scale=1.0):
            return torch.randn(*s, generator=g, device="cuda") * scale
        self.D, self.E, self.N, self.K, self.dt = D, E, N, 4, dtype
        self.w_in, self.w_out = r(D, 2 * E, scale=D ** -0.5).to(dtype), r(E, D, scale=E ** -0.5).to(dtype)
        self.w_bc, self.w_delta = r(E, 2 * N, scale=E ** -0.5).to(dtype), r(E, E, scale=E ** -0.5).to(dtype)
        self.p = {"taps": r(S, 4, E, scale=0.5), "bias": r(S, E, scale=0.1), "A": -torch.rand(S, E, N, generator=g, device="cuda") - 0.1,
                  "skip": r(S, E), "delta_bias": r(S, E) - 1, "w_post": 1 + r(S, D, scale=0.1), "scale": r(S, D, scale=0.3),
                  "w_pre": 1 + r(S, D, scale=0.1), "w_first": 1 + r(S, D, scale=0.1)}
        self.g = g

    def forward(self, x, ops, state=None, lengths=None):
        """x [R, T, D] fp32 residual; returns (residual, normed).  state: (window, h), moved."""
        R, T, D = x.shape
        p, dt = self.p, self.dt
        n = ops.norm(x.reshape(-1, D), None, p["w_first"], None, None)[1].reshape(R, T, D)
        ug = n @ self.w_in
        u, z = ug[..., :self.E], ug[..., self.E:]               # strided views
        u = ops.conv(u, p["taps"], p["bias"], state, lengths)
        bc = u @ self.w_bc
        B, C = bc[..., None, :self.N], bc[..., None, self.N:]
        y = ops.scan(u, u @ self.w_delta, p["A"], B, C, p["skip"], z, p["delta_bias"], state, lengths)
        o = y @ self.w_out
        x, n = ops.norm(x.reshape(-1, D), o.reshape(-1, D), p["w_pre"], p["w_post"], p["scale"])
        return x.reshape(R, T, D), n.reshape(R, T, D)


class Ours:
    def __init__(self, dt):
        self.dt = dt

    def norm(self, x, o, w_pre, w_post, scale):
        xo = torch.empty_like(x)
        no = torch.empty(x.shape, dtype=self.dt, device="cuda")
        zo.zo_block_norm(x, x_out=xo, n_out=no, o=o, w_post=w_post, scale=scale, w_pre=w_pre)
        return xo, no

    def conv(self, x, w, b, state, lengths):
        out = torch.empty(x.shape, dtype=x.dtype, device="cuda")
        if state is not None and x.shape[1] == 1:
            zo.zo_conv_step(x[:, 0], w, state[0], out[:, 0], bias=b)
        else:
            st = None if state is None else state[0]
            zo.zo_conv(x, w, out, bias=b, lengths=lengths, state_in=st, state_out=st)
        return out

    def scan(self, u, dl, A, B, C, skip, z, bias, state, lengths):
        out = torch.empty(u.shape, dtype=u.dtype, device="cuda")
        kw = dict(skip=skip, delta_bias=bias)
        if state is not None and u.shape[1] == 1:
            zo.zo_scan_step(u[:, 0], dl[:, 0], A, B[:, 0], C[:, 0], state[1], out[:, 0], z=z[:, 0], **kw)
        else:
            st = None if state is None else state[1]
            zo.zo_scan(u, dl, A, B, C, out, z=z, lengths=lengths, state_in=st, state_out=st, **kw)
        return out


class Reference:
    """The same in 64 bits, with every step's output rounded to its type."""

    def __init__(self, dt):
        self.dt = dt

    def norm(self, x, o, w_pre, w_post, scale):
        xo, n = ref.norm(x, o, None, w_post, scale, w_pre)
        return xo.to(x.dtype), n.to(self.dt)

    def conv(self, x, w, b, state, lengths):
        assert state is None
        return ref.conv(x, w, b, True, lengths)[0].to(x.dtype)

    def scan(self, u, dl, A, B, C, skip, z, bias, state, lengths):
        return ref.scan(u, dl, A, B, C, skip, z, bias, True, lengths)[0].to(u.dtype)


@gpu
def test_a_block_of_them_matches_the_reference():
    R, T, D, S = 6, 11, 32, 3
    b = Block(D, 48, 8, S, torch.float32, 1)
    x = torch.randn(R, T, D, generator=b.g, device="cuda")
    n = torch.tensor([11, 0, 3, 7, 1, 11], dtype=torch.int32, device="cuda")
    torch.backends.cuda.matmul.allow_tf32 = False
    got, want = b.forward(x, Ours(b.dt), lengths=n), b.forward(x, Reference(b.dt), lengths=n)
    for g, w in zip(got, want):
        # fp32 throughout: five operators and four products of 32..96 terms, all of order 1
        assert torch.allclose(g, w, rtol=2e-5, atol=2e-5)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tokens_one_by_one_give_the_prompt(dtype):
    R, T, D = 3, 10, 64
    b = Block(D, 64, 16, 1, dtype, 2)
    x = torch.randn(R, T, D, generator=b.g, device="cuda")
    ops = Ours(dtype)
    whole, _ = b.forward(x, ops)
    state = (torch.zeros(R, 3, 64, dtype=dtype, device="cuda"), torch.zeros(R, 64, 16, device="cuda"))
    first, _ = b.forward(x[:, :4].contiguous(), ops, state)         # a prompt of 4, then tokens
    rest = [b.forward(x[:, t:t + 1].contiguous(), ops, state)[0] for t in range(4, T)]
    got = torch.cat([first, *rest], 1)
    # the products' shapes differ, so their sums' order may: a rounding step of o either way
    tol = 32 * torch.finfo(dtype).eps
    assert torch.allclose(got, whole, rtol=tol, atol=tol)


@gpu
def test_probe_losses_of_a_block_in_one_call():
    """CD-RGE on the block's small parameters: 2 n perturbed copies as parameter sets, all in one
    call, against one call per copy; and the coefficients from their losses."""
    n, Bt, T, D, eps = 5, 4, 10, 32, 1e-2
    one = Block(D, 32, 8, 1, torch.float32, 3)
    x = torch.randn(Bt, T, D, generator=one.g, device="cuda")
    target = torch.randn(Bt, T, D, generator=one.g, device="cuda")
    ops = Ours(torch.float32)
    signs = {k: (torch.randint(0, 2, (n, *v.shape[1:]), generator=one.g, device="cuda") * 2 - 1).float()
             for k, v in one.p.items()}
    base = dict(one.p)
    one.p = {k: torch.cat([base[k] + s * eps * signs[k] for s in (1, -1)]) for k in base}
    out, _ = one.forward(x.repeat(2 * n, 1, 1), ops)
    losses = (out - target.repeat(2 * n, 1, 1)).square().reshape(2 * n, -1).mean(1)
    for i in range(2 * n):
        one.p = {k: base[k] + (1 if i < n else -1) * eps * signs[k][i % n:i % n + 1] for k in base}
        alone = (one.forward(x, ops)[0] - target).square().mean()
        # the same kernels on the same values; only the mean's order and the projections' tiles differ
        assert abs(float(losses[i]) - float(alone)) <= 1e-5 * float(alone)
    with zo.Context(10, 16, 32, 1, "f32", 1, 1, 0) as ctx:
        c = torch.empty(n, device="cuda")
        zo.zo_coeffs(ctx, losses[:n].contiguous(), losses[n:].contiguous(), n, eps, eps, c)
        assert torch.allclose(c, (losses[:n] - losses[n:]) / (2 * n), rtol=1e-4, atol=1e-7)


def training(seed, R, T, D, N):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def r(*s):
        return torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    u, dl, z, dout = (r(R, T, D) for _ in range(4))
    B, C = r(R, T, 1, N), r(R, T, 1, N)
    A, skip = -torch.rand(D, N, generator=g, device="cuda"), torch.randn(D, generator=g, device="cuda")
    w, bias = torch.randn(4, D, generator=g, device="cuda"), torch.randn(D, generator=g, device="cuda")
    got = {k: torch.empty_like(u) for k in ("x", "out", "du", "dd", "dz", "dx", "xn", "n", "dxn")}
    got |= {"dB": torch.empty_like(B), "dC": torch.empty_like(C), "dA": torch.empty_like(A), "dskip": torch.empty_like(skip),
            "dw": torch.empty_like(w), "db": torch.empty_like(bias), "dwp": torch.empty_like(bias)}
    kept = torch.empty(zo.zo_scan_checkpoint_shape(u.shape, N), device="cuda")

    def call(stream=None):
        k = dict(stream=stream)
        zo.zo_conv(u, w, got["x"], bias=bias, **k)
        zo.zo_scan(got["x"], dl, A, B, C, got["out"], skip=skip, z=z, checkpoints=kept, **k)
        zo.zo_block_norm(got["out"].view(-1, D), n_out=got["n"].view(-1, D), w_pre=bias, **k)
        zo.zo_block_norm_backward(got["out"].view(-1, D), dn=dout.view(-1, D), dx=got["dxn"].view(-1, D), w_pre=bias, dw_pre=got["dwp"], **k)
        zo.zo_scan_backward(got["x"], dl, A, B, C, got["dxn"], kept, got["du"], got["dd"], got["dA"], got["dB"], got["dC"],
                            skip=skip, dskip=got["dskip"], z=z, dz=got["dz"], **k)
        zo.zo_conv_backward(u, w, got["du"], got["dx"], got["dw"], bias=bias, dbias=got["db"], **k)
    got.pop("xn")
    return call, got, u


SIZES = [(2, 40, 64, 16), (1, 3000, 32, 8)]


@gpu
@pytest.mark.parametrize("size", SIZES)
def test_results_are_the_same_each_time(size):
    call, got, _ = training(1, *size)
    call()
    first = {k: v.clone() for k, v in got.items()}
    for _ in range(3):
        for v in got.values():
            v.fill_(float("nan"))
        call()
        for k, v in got.items():
            assert torch.equal(v, first[k]), k


@gpu
@pytest.mark.parametrize("size", SIZES)
def test_two_streams_at_once(size):
    calls = [training(s, *size) for s in (1, 2)]
    want = []
    for call, got, _ in calls:
        call()
        want.append({k: v.clone() for k, v in got.items()})
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _, got, _ in calls:
        for v in got.values():
            v.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(5):
        calls[0][0](streams[0])                      # given
        with torch.cuda.stream(streams[1]):          # current
            calls[1][0]()
    torch.cuda.synchronize()
    for (_, got, _), w in zip(calls, want):
        for k in w:
            assert torch.equal(got[k], w[k]), k


@gpu
@pytest.mark.parametrize("size", SIZES)
def test_captured_graphs_replay_with_new_inputs(size):
    pairs = []
    for s in (1, 2):                                 # two graphs, replayed at once
        call, got, u = training(s, *size)
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        pairs.append((graph, call, got, u))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _, _, _, u in pairs:
        u.copy_(torch.randn(u.shape, device="cuda"))
    torch.cuda.synchronize()
    for (graph, _, _, _), st in zip(pairs, streams):
        with torch.cuda.stream(st):
            for _ in range(4):
                graph.replay()
    torch.cuda.synchronize()
    for _, call, got, _ in pairs:
        replayed = {k: v.clone() for k, v in got.items()}
        call()
        for k, v in got.items():
            assert torch.equal(v, replayed[k]), k


@gpu
def test_given_workspaces():
    call, got, _ = training(3, 1, 3000, 32, 8)
    x = torch.randn(2, 50, 24, device="cuda")
    w, dw, dx = torch.randn(4, 24, device="cuda"), torch.empty(4, 24, device="cuda"), torch.empty_like(x)
    zo.zo_conv_backward(x, w, x, dx, dw)
    want = dw.clone()
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
    zo.zo_conv_backward(x, w, x, dx, dw, workspace=ws)
    assert torch.equal(dw, want)
    with pytest.raises(zo.ZOError):
        zo.zo_conv_backward(x, w, x, dx, dw, workspace=ws[:64])
    with pytest.raises(ValueError):
        zo.zo_conv_backward(x, w, x, dx, dw, workspace=ws.cpu())


@gpu
def test_offsets_beyond_32_bits():
    """Rows more than 2^31 elements apart, and a state cache of such rows."""
    D, N, far = 64, 16, 2 ** 31 + 64
    flat = torch.empty(far + 8 * D, dtype=torch.bfloat16, device="cuda")
    x = flat.as_strided((2, 8, D), (far, D, 1))
    near = torch.randn(2, 8, D, device="cuda").to(torch.bfloat16)
    x.copy_(near)
    w = torch.randn(4, D, device="cuda")
    a, b = torch.empty_like(near), torch.empty_like(near)
    zo.zo_conv(x, w, a)
    zo.zo_conv(near, w, b)
    assert torch.equal(a, b)
    A, B = -torch.rand(D, N, device="cuda"), torch.randn(2, 8, 1, N, device="cuda").to(torch.bfloat16)
    zo.zo_scan(x, near, A, B, B, a)
    zo.zo_scan(near, near, A, B, B, b)
    assert torch.equal(a, b)
    del flat, x
    cache = torch.empty(far + D * N, device="cuda").as_strided((2, D, N), (far, N, 1))
    h = torch.randn(2, D, N, device="cuda")
    cache.copy_(h)
    ya, yb = torch.empty(2, D, device="cuda"), torch.empty(2, D, device="cuda")
    f = near.float()
    zo.zo_scan_step(f[:, 0], f[:, 1], A, B[:, 0].float(), B[:, 1].float(), cache, ya)
    zo.zo_scan_step(f[:, 0], f[:, 1], A, B[:, 0].float(), B[:, 1].float(), h, yb)
    assert torch.equal(ya, yb) and torch.equal(cache, h)


@gpu
def test_shared_parameters_and_broadcast_inputs():
    """A and the taps shared by all sets while other parameters differ; B and C of one row for all."""
    g = torch.Generator(device="cuda")
    g.manual_seed(9)

    def r(*s):
        return torch.randn(*s, generator=g, device="cuda")
    R, T, D, N, S, K = 6, 20, 24, 8, 3, 4
    u, dl, dout = r(R, T, D), r(R, T, D), r(R, T, D)
    A, bias, skip = -torch.rand(D, N, generator=g, device="cuda"), r(S, D), r(D)
    B, C = r(1, T, 1, N).expand(R, T, 1, N), r(R, 1, 1, N).expand(R, T, 1, N)
    kept = torch.empty(zo.zo_scan_checkpoint_shape(u.shape, N), device="cuda")

    def both(A, skip, B, C):
        out, du, dd = (torch.empty_like(u) for _ in range(3))
        dA, ds, db = torch.empty(S, D, N, device="cuda"), torch.empty(S, D, device="cuda"), torch.empty(S, D, device="cuda")
        dB, dC = (torch.empty(R, T, 1, N, device="cuda") for _ in range(2))
        zo.zo_scan(u, dl, A, B, C, out, skip=skip, delta_bias=bias, checkpoints=kept)
        zo.zo_scan_backward(u, dl, A, B, C, dout, kept, du, dd, dA, dB, dC, skip=skip, dskip=ds, delta_bias=bias,
                            ddelta_bias=db)
        return out, du, dd, dA, ds, db, dB, dC
    for a, b in zip(both(A, skip, B, C), both(A.expand(S, D, N).contiguous(), skip.expand(S, D).contiguous(),
                                              B.contiguous(), C.contiguous())):
        assert torch.equal(a, b)
    w, cb, a, b = r(K, D), r(S, D), torch.empty_like(u), torch.empty_like(u)
    zo.zo_conv(u, w, a, bias=cb)
    zo.zo_conv(u, w.expand(S, K, D).contiguous(), b, bias=cb)
    assert torch.equal(a, b)
    x, o = u.reshape(-1, D), dl.reshape(-1, D)
    zo.zo_block_norm(x, x_out=a.view(-1, D), o=o, w_post=skip, scale=cb)
    zo.zo_block_norm(x, x_out=b.view(-1, D), o=o, w_post=skip.expand(S, D).contiguous(), scale=cb)
    assert torch.equal(a, b)


@gpu
def test_steps_without_state_out_leave_the_state():
    R, D, N, K = 3, 16, 8, 4
    u, st = torch.randn(R, D, device="cuda"), torch.randn(R, D, N, device="cuda")
    A, B = -torch.rand(D, N, device="cuda"), torch.randn(R, 1, N, device="cuda")
    out, want, kept = torch.empty_like(u), torch.empty_like(u), st.clone()
    zo.zo_scan_step(u, u, A, B, B, st.clone(), want)
    t, bc = (lambda p: block._Tensor(p.data_ptr(), D, 0)), block._Tensor(B.data_ptr(), N, 0)
    a = block.ScanArgs(R, 1, D, 1, N, 1, zo.ZO_DTYPE_FP32, zo.ZO_SCAN_SOFTPLUS, t(u), t(u), t(out), block._Tensor(), bc, bc,
                       block._F32(A.data_ptr(), 0))
    a.state_in = block._F32(st.data_ptr(), D * N)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert zo.load_library().zo_scan_step(a, stream) == zo.ZO_OK
    assert torch.equal(out, want) and torch.equal(st, kept)
    win, w = torch.randn(R, K - 1, D, device="cuda"), torch.randn(K, D, device="cuda")
    kept = win.clone()
    zo.zo_conv_step(u, w, win.clone(), want)
    a = block.ConvArgs(R, 1, D, K, 1, zo.ZO_DTYPE_FP32, zo.ZO_CONV_SILU, t(u), t(out), block._F32(w.data_ptr(), 0))
    a.state_in = block._Tensor(win.data_ptr(), (K - 1) * D, D)
    assert zo.load_library().zo_conv_step(a, stream) == zo.ZO_OK
    assert torch.equal(out, want) and torch.equal(win, kept)
