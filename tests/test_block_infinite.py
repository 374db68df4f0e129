"""Infinite inputs of the selective scan: where the formula gives an infinity of one sign, so do the
kernels, whatever number of states a lane of theirs is made for; other channels and earlier steps
stay as they are."""
import pytest
import torch

import zero_order_recurrent_b200 as zo
from tests import block_reference as ref

pytestmark = pytest.mark.gpu
INF = float("inf")
STATES = [1, 2, 3, 4, 5, 7, 8, 9, 12, 13, 16, 18, 20, 24, 31, 33, 64, 100, 128]


@pytest.fixture(scope="module", autouse=True)
def library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from zero_order_recurrent_b200 import build
    build.build()
    zo.load_library()


def inputs(R, T, D, N, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(N)

    def r(*s):
        return 0.5 + torch.rand(*s, generator=g, device="cuda")
    u, dl, z, dout = (r(R, T, D).to(dtype) for _ in range(4))
    B, C = (r(R, T, 1, N).to(dtype) for _ in range(2))
    return u, dl, z, dout, -0.2 * r(D, N), B, C


def same(got, want):
    """Equal infinities at the same places; elsewhere finite and near (that part is other tests')."""
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf].double(), want[inf])
    assert not torch.isnan(got).any()
    assert torch.allclose(got[~inf].double(), want[~inf], rtol=0.02, atol=0.02)


# the channel's input at a step, or its time step, infinite; one pass over time, and parts of it
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,T", [(700, 6), (2, 6), (1, 70)])
@pytest.mark.parametrize("N", STATES)
def test_infinite_inputs_give_infinite_outputs(N, R, T, dtype):
    D = 6
    u, dl, z, _, A, B, C = inputs(R, T, D, N, dtype)
    u[0, 2, 1], u[0, 4, 3], dl[R - 1, 3, 5] = INF, -INF, INF
    out, so = torch.empty_like(u), torch.empty(R, D, N, device="cuda")
    zo.zo_scan(u, dl, A, B, C, out, z=z, softplus=False, state_out=so)
    want, last, _, _ = ref.scan(u, dl, A[None], B, C, z=z, softplus=False)
    assert torch.isinf(want).sum() == T - 2 + T - 4 + T - 3
    same(out, want)
    same(so, last)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,D", [(3, 6), (1500, 256)])
@pytest.mark.parametrize("N", STATES)
def test_infinite_inputs_of_single_tokens(N, R, D, dtype):
    u, dl, z, _, A, B, C = inputs(R, 1, D, N, dtype)
    u[0, 0, 1], u[1, 0, 3], dl[R - 1, 0, 5] = INF, -INF, INF
    out, st = torch.empty_like(u[:, 0]), torch.ones(R, D, N, device="cuda")
    want, last, _, _ = ref.scan(u, dl, A[None], B, C, z=z, softplus=False, state=st)
    zo.zo_scan_step(u[:, 0], dl[:, 0], A, B[:, 0], C[:, 0], st, out, z=z[:, 0], softplus=False)
    same(out, want[:, 0])
    same(st, last)


@pytest.mark.parametrize("skip", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [6, 70])
@pytest.mark.parametrize("N", STATES)
def test_infinite_inputs_and_gradients(N, T, dtype, skip):
    """With everything positive the gradients are infinite, finite or (where terms differ in sign, or
    an infinity meets the first step's state 0) NaN, as the formulas are."""
    R, D = 2, 6
    u, dl, z, dout, A, B, C = inputs(R, T, D, N, dtype)
    u[0, 2, 1], u[0, 4, 3] = INF, INF
    dout[1, 3, 2] = INF
    sk = torch.ones(D, device="cuda") if skip else None
    ds = torch.empty(D, device="cuda") if skip else None
    kept = torch.empty(zo.zo_scan_checkpoint_shape(u.shape, N), device="cuda")
    zo.zo_scan(u, dl, A, B, C, torch.empty_like(u), skip=sk, z=z, softplus=False, checkpoints=kept)
    du, dd, dz, dB, dC, dA = (torch.empty_like(t) for t in (u, dl, z, B, C, A))
    zo.zo_scan_backward(u, dl, A, B, C, dout, kept, du, dd, dA, dB, dC, skip=sk, dskip=ds, z=z, dz=dz, softplus=False)
    want = ref.scan_backward(u, dl, A[None], B, C, dout, skip=None if sk is None else sk[None], z=z, softplus=False)
    if not skip:  # the reference has a skip of 0 there
        assert torch.isnan(want["du"]).nonzero().tolist() == [[1, 3, 2]]
        want["du"][1, 3, 2] = INF
    else:
        assert torch.isinf(ds).tolist() == [False, True, True, True, False, False]
    assert torch.isinf(want["dz"]).sum() == T - 2 + T - 4 + 1 and torch.isinf(want["ddelta"]).any()
    for got, k in ((du, "du"), (dd, "ddelta"), (dz, "dz"), (dB, "dB"), (dC, "dC"), (dA[None], "dA")):
        there = ~torch.isnan(want[k])
        assert torch.equal(torch.isnan(got), ~there), k
        same(got[there], want[k][there])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R", [1, 700])
def test_infinities_outlast_decays_that_vanish_together(R, dtype):
    """No step's decay is 0, but those of 32 steps together are below fp32: an infinite state, and an
    infinite gradient, stay infinite over them, whether or not time is divided there."""
    T, D, N = 140, 6, 8
    u, _, z, dout, _, B, C = inputs(R, T, D, N, dtype)
    dl, A = torch.full_like(u, 5.0), torch.full((D, N), -4.0, device="cuda")   # e^-20 a step
    u[0, 3, 1] = INF
    st, so = torch.ones(R, D, N, device="cuda"), torch.empty(R, D, N, device="cuda")
    st[0, 4, 2] = INF
    out, kept = torch.empty_like(u), torch.empty(zo.zo_scan_checkpoint_shape(u.shape, N), device="cuda")
    zo.zo_scan(u, dl, A, B, C, out, z=z, softplus=False, state_in=st, state_out=so, checkpoints=kept)
    want, last, _, _ = ref.scan(u, dl, A[None], B, C, z=z, softplus=False, state=st)
    assert torch.isinf(want[0]).sum() == T - 3 + T and torch.isinf(last[0]).sum() == N + 1
    same(out, want)
    same(so, last)

    u[0, 3, 1], st[0, 4, 2] = 1, 1
    dso, dsi = torch.ones_like(st), torch.empty_like(st)
    dso[0, 4, 2], dout[0, T - 2, 1] = INF, INF
    zo.zo_scan(u, dl, A, B, C, out, z=z, softplus=False, state_in=st, checkpoints=kept)
    du, dd, dz, dB, dC, dA = (torch.empty_like(t) for t in (u, dl, z, B, C, A))
    zo.zo_scan_backward(u, dl, A, B, C, dout, kept, du, dd, dA, dB, dC, z=z, dz=dz, softplus=False, dstate_out=dso,
                        dstate_in=dsi)
    want = ref.scan_backward(u, dl, A[None], B, C, dout, z=z, softplus=False, state=st, dstate=dso)
    assert torch.isinf(want["dstate_in"][0]).sum() == N + 1
    want["du"][0, T - 2, 1] = INF  # (the reference has a skip of 0 there)
    for got, k in ((du, "du"), (dB, "dB"), (dC, "dC"), (dz, "dz"), (dsi, "dstate_in"), (dA[None], "dA")):
        same(got, want[k])
