"""Slow decays of the selective scan: what the errors of the exponentials add up to over a state's
memory, which the bounds per step of the other tests leave room for.

M = 1 / (rate * step) steps is a state's memory.  All inputs are positive and the steps vary, so
the state has no cancellation and its roundings are independent of one another.  A step's roundings,
in units of u = 2^-24 relative to the state: that of the decay, between 1/2 and 1, is half a step
of 2^-24, so 0.29 in the root mean square; that of the new state 0.58 at most; together 0.65.
Over the memory they add up to 0.65 sqrt(M / 2) = 0.46 sqrt(M), and the bound takes sqrt(M).  What
is the same at every step: the rate's product with log2(e) and that constant, 1 each of the
exponent, which over the memory is 1; the polynomial for decays near 1, 0.05 a step where the
memory is under 12 steps and 0.002 else.  4 for these together."""
import pytest
import torch

import zero_order_recurrent_b200 as zo
from tests import block_reference as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F64 = torch.float64
STEPS = [2.0 ** -12, 2.0 ** -10, 2.0 ** -9, 2.0 ** -8, 2.0 ** -7, 2.0 ** -6, 2.0 ** -4]


@pytest.fixture(scope="module", autouse=True)
def library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from zero_order_recurrent_b200 import build
    build.build()
    zo.load_library()


def inputs(R, T, D, N, step, dtype=torch.float32, seed=0):
    """u, delta, A, B, C: rates 1..2, steps from 0.5 to 1.5 of `step`, everything else 0.5..1.5."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def r(*s):
        return 0.5 + torch.rand(*s, generator=g, device="cuda")
    u, B, C = (r(*s).to(dtype) for s in ((R, T, D), (R, T, 1, N), (R, T, 1, N)))
    return u, (step * r(R, T, D)).to(dtype), -(0.5 + r(D, N)), B, C


def bound(step, dtype):
    M = 1 / step
    tol = U * (M ** 0.5 + 4)
    if dtype is not torch.float32:
        # the special function unit's own results, at most 2e-8 too small on average for decays up
        # to 2^-9 below 1 and right on average beyond (csrc/k_scan.cuh)
        tol += 2e-8 * min(M, 512)
    return tol


def last_state(u, delta, A, B, st):
    """sum_t exp(A (sum of the later steps)) d_t u_t B_t, in 64 bits."""
    d = delta.to(F64)
    later = d.flip(1).cumsum(1).flip(1) - d
    out = []
    for r in range(u.shape[0]):
        w = torch.exp(later[r, :, :, None] * A.to(F64)) * (d[r] * u[r].to(F64))[..., None] * B[r].to(F64)
        out.append(w.sum(0) + torch.exp(d[r].sum(0)[:, None] * A.to(F64)) * st[r].to(F64))
    return torch.stack(out)


def check(got, want, tol):
    off = ((got.double() - want) / want).square().mean().sqrt()
    assert off <= tol, (float(off), tol)


# one pass over time, and few rows and channels, whose time is divided
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,D", [(1, 8), (700, 8)])
@pytest.mark.parametrize("step", STEPS)
def test_states(step, R, D, dtype):
    N, T = 8, min(4096, int(4 / step)) if R > 1 else int(4 / step)
    u, dl, A, B, C = inputs(R, T, D, N, step, dtype)
    a = zo.block.ScanArgs(R, T, D, 1, N, 1, 0, 0)
    assert (zo.load_library().zo_scan_workspace(a) > 0) == (R == 1 and T > 32)
    st = torch.rand(R, D, N, device="cuda") + 0.5
    out, so = torch.empty_like(u), torch.empty_like(st)
    zo.zo_scan(u, dl, A, B, C, out, softplus=False, state_in=st, state_out=so)
    check(so, last_state(u, dl, A, B, st), bound(step, dtype))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("step", [2.0 ** -10, 2.0 ** -8, 2.0 ** -6])
@pytest.mark.parametrize("N", [16, 7])
def test_single_tokens(step, N, dtype):
    R, T, D = 2, int(2 / step), 64
    u, dl, A, B, C = inputs(R, T, D, N, step, dtype)
    st = torch.rand(R, D, N, device="cuda") + 0.5
    want = last_state(u, dl, A, B, st)
    y = torch.empty(R, D, dtype=dtype, device="cuda")
    for t in range(T):
        zo.zo_scan_step(u[:, t], dl[:, t], A, B[:, t], C[:, t], st, y, softplus=False)
    check(st, want, bound(step, dtype))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("step", STEPS)
def test_carries(step, dtype):
    """The gradient that arrives at the first state, through all of time (divided in parts)."""
    R, T, D, N = 1, int(4 / step), 8, 8
    u, dl, A, B, C = inputs(R, T, D, N, step, dtype)
    dout, ds = (0.5 + torch.rand(R, T, D, device="cuda")).to(dtype), torch.rand(R, D, N, device="cuda") + 0.5
    kept = torch.empty(zo.zo_scan_checkpoint_shape(u.shape, N), device="cuda")
    out, g0 = torch.empty_like(u), torch.empty_like(ds)
    zo.zo_scan(u, dl, A, B, C, out, softplus=False, checkpoints=kept)
    du, dd, dA, dB, dC = (torch.empty_like(t) for t in (u, dl, A, B, C))
    zo.zo_scan_backward(u, dl, A, B, C, dout, kept, du, dd, dA, dB, dC, softplus=False, dstate_out=ds, dstate_in=g0)
    d = dl.to(F64)
    w = torch.exp(d.cumsum(1)[..., None] * A.to(F64)) * (dout.to(F64)[..., None] * C.to(F64))
    want = w.sum(1) + torch.exp(d.sum(1)[..., None] * A.to(F64)) * ds.to(F64)
    check(g0, want, bound(step, dtype))


@pytest.mark.parametrize("step", [2.0 ** -10, 2.0 ** -8, 2.0 ** -6])
@pytest.mark.parametrize("R,D", [(1, 8), (700, 8)])
def test_rate_gradients(step, R, D):
    """dA sums T products of a carry and a state (and R rows): both have the bound above, and the sum,
    in partial sums of at most 1024 steps, a rounding of up to u / 2 a step: sqrt(1024) / 2."""
    T, N = 1024, 8
    u, dl, A, B, C = inputs(R, T, D, N, step)
    dout = 0.5 + torch.rand(R, T, D, device="cuda")
    kept = torch.empty(zo.zo_scan_checkpoint_shape(u.shape, N), device="cuda")
    zo.zo_scan(u, dl, A, B, C, torch.empty_like(u), softplus=False, checkpoints=kept)
    du, dd, dA, dB, dC = (torch.empty_like(t) for t in (u, dl, A, B, C))
    zo.zo_scan_backward(u, dl, A, B, C, dout, kept, du, dd, dA, dB, dC, softplus=False)
    want = ref.scan_backward(u, dl, A[None], B, C, dout, softplus=False)["dA"][0]
    check(dA, want, 2 * bound(step, torch.float32) + 16 * U)
