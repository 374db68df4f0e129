"""The forms of the state-space block's kernels that sizes choose between, each on sizes that choose
it, and the gradients by the size of their error as a whole.

Bound of a gradient as a whole.  Its terms have random signs, and so do their roundings: a sum of K
terms of size a is about a sqrt(K), and so is the error of terms that are each off by e: e relative
to the sum.  e is the error of a state and of a carry, u = 2^-24 times sqrt(M) + 4 each for a memory
of M steps (tests/test_block_decays.py), here at most 4 steps or, where decays are random down to 1,
T <= 2500 of them for a few states: 2 (50 + 4) u; about ten more operations.  The sums run over at most
1024 steps in one register, whose running value has the size a sqrt(k): a rounding of up to u / 2
of it at each step k is u / 2 a sqrt(K^2 / 2), relative to a sqrt(K) u sqrt(K / 8) = 12 u; the
partial sums, K of them, likewise.  Together under (128 + sqrt(R T)) u, and the output's own rounding."""
import pytest
import torch

import zero_order_recurrent_b200 as zo
from tests import block_reference as ref
from tests.test_block_gpu import DT, SCAN, U, near, poison, scan_inputs, scan_ops
from zero_order_recurrent_b200 import block

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    from zero_order_recurrent_b200 import build
    build.build()
    zo.load_library()


def backward_workspace(R, T, D, G, N, S):
    return zo.load_library().zo_scan_backward_workspace(block.ScanArgs(R, T, D, G, N, S, zo.ZO_DTYPE_FP32, 0))


def planned(R, T, D, G, N, tiles, parts, flushes):
    """The workspace of a backward pass with these channel tiles of a group, parts of time and partial
    sums of a part: partial dB and dC, partial dA, dskip and ddelta_bias, carries and sums of steps."""
    bc = tiles * R * T * G * 2 * N
    param = R * parts * flushes * (D * N + 2 * D)
    carries = (-(-R * parts * D * N // 4) * 4 + R * parts * D) if parts > 1 else 0
    return 4 * (bc + param + carries)


# R, T, D, G, N, S, dtype, ragged, state, gate, softplus, pad and the plan: channel tiles of a group (of
# several warps, but for the last three), parts of time, partial sums of a part
BACK = [
    ((2, 40, 128, 1, 16, 1, "bf16", True, True, True, True, False), (1, 2, 1)),
    ((3, 33, 250, 1, 16, 3, "f32", True, True, True, True, False), (2, 2, 1)),
    ((600, 9, 250, 1, 16, 2, "bf16", True, True, False, True, False), (2, 1, 1)),
    ((2, 40, 256, 2, 12, 1, "f16", True, True, True, True, True), (1, 2, 1)),
    ((2, 70, 128, 1, 8, 1, "f32", True, True, True, True, False), (1, 3, 1)),
    ((4, 35, 500, 2, 5, 2, "bf16", None, False, True, False, False), (2, 2, 1)),
    ((2, 50, 64, 1, 24, 1, "f32", True, True, True, True, False), (1, 2, 1)),
    ((300, 20, 120, 1, 24, 1, "f32", True, False, True, True, False), (2, 1, 1)),
    ((2, 40, 32, 1, 64, 1, "bf16", True, True, True, True, False), (1, 2, 1)),
    ((2, 40, 31, 1, 100, 1, "f32", True, True, True, True, False), (2, 2, 1)),
    ((900, 1100, 8, 1, 16, 1, "f32", None, False, False, True, False), (1, 1, 2)),
    ((900, 2100, 8, 1, 4, 2, "bf16", True, False, True, True, False), (1, 1, 3)),
    ((1, 5000, 16, 1, 16, 1, "f32", None, True, True, True, False), (1, 157, 1)),
]


@pytest.mark.parametrize("case,plan", BACK)
def test_plans(case, plan):
    R, T, D, G, N, S = case[:6]
    assert backward_workspace(R, T, D, G, N, S) == planned(R, T, D, G, N, *plan)


def gradients(case, seed=3):
    """The kernel's and the reference's gradients by name, and the reference's inputs."""
    R, T, D, G, N, S, dtype, ragged, state, gate, softplus, pad = case
    i, n, u, dl, A, B, C, kw, bias, st = scan_inputs(*case, seed)
    dt = u.dtype
    dout = poison(i.act(R, T, D, dtype=dt), n)
    kept = torch.empty(zo.zo_scan_checkpoint_shape(u.shape, N), device="cuda")
    zo.zo_scan(u, dl, A, B, C, torch.empty_like(u), delta_bias=bias, softplus=softplus, lengths=n, state_in=st,
               checkpoints=kept, **kw)

    def new(*s, dtype=torch.float32):
        return torch.full(s, float("nan"), dtype=dtype, device="cuda")
    got = {k: new(R, T, D, dtype=dt) for k in ("du", "ddelta") + (("dz",) if gate else ())}
    got |= {k: new(R, T, G, N, dtype=dt) for k in ("dB", "dC")}
    got |= {"dA": new(S, D, N), "dskip": new(S, D), "ddelta_bias": new(S, D)}
    dso = i.normal(R, D, N) if state else None
    if state:
        got["dstate_in"] = new(R, D, N)
    zo.zo_scan_backward(u, dl, A, B, C, dout, kept, delta_bias=bias, softplus=softplus, lengths=n, dstate_out=dso,
                        **got, **kw)
    args = (u, dl, A, B, C, dout, kw["skip"], kw["z"], bias, softplus, n, st, dso)
    return got, args, n


def tolerance(got, R, T):
    return torch.finfo(got.dtype).eps / 2 + (128 + (R * T) ** 0.5) * U


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


@gpu
@pytest.mark.parametrize("case", [c for c, _ in BACK] + SCAN)
def test_gradients_as_a_whole(case):
    R, T, D, G, N, S = case[:6]
    got, args, n = gradients(case)
    want, size = ref.scan_backward(*args), None
    for k, v in got.items():
        if want[k].norm() == 0:  # a single row of length 0
            assert not v.any(), k
            continue
        tol = tolerance(v, R, T)
        assert off(v, want[k]) <= tol, (k, off(v, want[k]), tol)
        # what the bound is worth: nothing, half, and a sum without one row are far outside
        assert min(off(torch.zeros_like(v), want[k]), off(v / 2, want[k])) > 4 * tol
    row = max(range(R), key=lambda r: T if n is None else int(n[r])) if R < 1000 else R - 1
    one = list(args)
    for at in (0, 1, 3, 4, 5, 7, 10, 11, 12):  # what has rows, and what has sets
        one[at] = None if one[at] is None else one[at][row:row + 1]
    for at in (2, 6, 8):
        one[at] = one[at][row // (R // S)][None]
    alone = ref.scan_backward(*one)
    s = row // (R // S)
    for k in ("dA", "dskip", "ddelta_bias"):
        if want[k].norm() == 0:  # one step from the state 0
            continue
        without = got[k].double().clone()
        without[s] -= alone[k][0]
        assert off(without, want[k]) > 4 * tolerance(got[k], R, T), k


def lanes(N):
    return 1 << max(0, (N - 1).bit_length() - 2)


# R, D, N, S: four rows a thread, which takes 4 * 148 * 2048 threads with one, and one; whole lanes,
# lanes without states, states one by one
STEP = [(R, -(-4 * 148 * 2048 // (R * lanes(N))) + 8, N, S) for N in (16, 12, 24, 7)
        for R, S in ((5, 1), (9, 3), (20, 5), (14, 2), (10, 10), (12, 3))] + \
       [(R, D, N, S) for N in (1, 4, 7, 8, 12, 16, 24, 128) for D in (5, 96) for R, S in ((1, 1), (6, 3), (7, 7))]


@gpu
@pytest.mark.parametrize("R,D,N,S", STEP)
def test_single_tokens(R, D, N, S):
    """Sets of 1, 3, 4, 5 and 7 rows, in place and not, with and without gate and skip; nothing behind
    the last row is touched."""
    for turn, dtype in enumerate(("bf16", "f32", "f16")):
        i, _, u, dl, A, B, C, kw, bias, st = scan_inputs(R, 1, D, 1, N, S, dtype, None, True, turn != 1, True, False, turn)
        if turn == 2:
            kw["skip"] = None
        z = kw.pop("z")
        args = (u, dl, A, B, C, kw["skip"], z, bias, True, None, st)
        (want, last, _, _), (size, slast, _, _) = ref.scan(*args), ref.scan(*args, size=True)
        ops = scan_ops(1, N, dl, A, bias, True)
        out = torch.full((R + 3, D), float("nan"), dtype=DT[dtype], device="cuda")
        new = torch.full((R + 3, D, N), float("nan"), device="cuda")
        now = new.clone()
        now[:R] = st
        call = dict(delta_bias=bias, z=None if z is None else z[:, 0], **kw)
        zo.zo_scan_step(u[:, 0], dl[:, 0], A, B[:, 0], C[:, 0], st, out[:R], state_out=new[:R], **call)
        near(out[:R], want[:, 0], size[:, 0], ops, "out")
        near(new[:R], last, slast, ops, "state")
        first = out.clone()
        zo.zo_scan_step(u[:, 0], dl[:, 0], A, B[:, 0], C[:, 0], now[:R], out[:R], **call)  # in place
        assert torch.equal(now[:R], new[:R]) and torch.equal(out[:R], first[:R])
        for t in (out, new, now):
            assert torch.isnan(t[R:]).all()


# ---- the norms' combinations ---------------------------------------------------------

@gpu
@pytest.mark.parametrize("gate_first", [False, True])
@pytest.mark.parametrize("given", range(16))
def test_norm_combinations(given, gate_first):
    """Every set of gate, norm after the block, residual scale and norm before the next, the plain
    x + o among them, forward and backward, against the reference in 64 bits."""
    names = [k for b, k in enumerate(("gate", "w_post", "scale", "w_pre")) if given >> b & 1]
    if gate_first and "gate" not in names:
        pytest.skip("no gate to put first")
    g = torch.Generator(device="cuda")
    g.manual_seed(given)
    for R, D, S in ((6, 264, 2), (5, 1000, 1), (4, 33, 4)):
        def r(*s):
            return torch.randn(*s, generator=g, device="cuda")
        x, p = r(R, D), {"o": r(R, D)}
        p |= {k: r(R, D) if k == "gate" else r(S, D) for k in names}
        kw = dict(eps=1e-5, gate_first=gate_first)
        xo, no = torch.empty_like(x), torch.empty_like(x) if "w_pre" in p else None
        zo.zo_block_norm(x, x_out=xo, n_out=no, **kw, **p)
        want, wn = ref.norm(x, **kw, **p)
        # the sums of D squares, off by D u at most, and a dozen operations
        tol = (D + 16) * U
        assert off(xo, want) <= tol and (no is None or off(no, wn) <= 2 * tol)
        dxo, dn = r(R, D), r(R, D) if "w_pre" in p else None
        got = {"dx": torch.empty_like(x)} | {"d" + k: torch.empty_like(v) for k, v in p.items()}
        zo.zo_block_norm_backward(xo, dn=dn, dx_out=dxo, **got, **kw, **p)
        wants = ref.norm_backward(xo, dn, dxo, **kw, **p)
        for k, v in got.items():
            assert off(v, wants[k]) <= 4 * tol, k


# ---- workspaces ------------------------------------------------------------------------

def test_norm_workspaces_of_all_sizes():
    lib = zo.load_library()
    for rows in (1, 2, 7, 100, 591, 592, 593, 5000, 2 ** 20):
        for channels in (1, 255, 256, 257, 512, 513, 1024, 1025, 2048, 2049, 4096, 4097, 8192, 8193, 16384):
            for sets in (1, 2, 5, 7, 100):
                if rows % sets:
                    continue
                n = lib.zo_block_norm_backward_workspace(block.NormArgs(rows, channels, sets, 0, 0, 0, 1e-5))
                groups = n // (12 * sets * channels)  # row groups of a set: three gradients each
                assert n == groups * 12 * sets * channels and 1 <= groups <= max(rows // sets + 3, 1)


@gpu
@pytest.mark.parametrize("what", ["scan", "scan_backward", "scan_backward_flushes", "norm_backward", "conv_backward"])
def test_given_workspaces_with_old_contents(what):
    """A workspace of exactly the size, full of NaN (0xFF): the same results, and nothing behind it."""
    case = {"scan_backward_flushes": (900, 1100, 8, 1, 16, 1)}.get(what, (1, 3000, 32, 1, 8, 1))
    R, T, D, G, N, S = case
    i, _, u, dl, A, B, C, kw, bias, st = scan_inputs(*case, "f32", None, True, True, True, False, 5)
    kept = torch.empty(zo.zo_scan_checkpoint_shape(u.shape, N), device="cuda")
    out = torch.empty_like(u)
    zo.zo_scan(u, dl, A, B, C, out, delta_bias=bias, state_in=st, checkpoints=kept, **kw)
    lib, sizes = zo.load_library(), block.ScanArgs(R, T, D, G, N, S, 0, 0)
    x, w, p = u[0], torch.randn(4, D, device="cuda"), {"o": dl[0], "gate": kw["z"][0], "w_post": bias, "scale": bias, "w_pre": bias}

    def run(ws):
        if what == "scan":
            got = [torch.empty_like(u), torch.empty_like(st)]
            zo.zo_scan(u, dl, A, B, C, got[0], delta_bias=bias, state_in=st, state_out=got[1], workspace=ws, **kw)
        elif what == "norm_backward":
            got = [torch.empty_like(x) for _ in range(3)] + [torch.empty_like(bias) for _ in range(3)]
            zo.zo_block_norm_backward(x, dl[0], u[0], *got, workspace=ws, **p)
        elif what == "conv_backward":
            got = [torch.empty_like(u), torch.empty_like(w), torch.empty_like(bias)]
            zo.zo_conv_backward(u, w, dl, got[0], got[1], bias=bias, dbias=got[2], workspace=ws)
        else:
            got = [torch.empty_like(t) for t in (u, dl, A, B, C, kw["skip"], kw["z"], bias)]
            zo.zo_scan_backward(u, dl, A, B, C, dl, kept, *got[:5], dskip=got[5], dz=got[6], delta_bias=bias,
                                ddelta_bias=got[7], workspace=ws, **kw)
        return got
    need = {"scan": lambda: lib.zo_scan_workspace(sizes), "scan_backward": lambda: lib.zo_scan_backward_workspace(sizes),
            "scan_backward_flushes": lambda: lib.zo_scan_backward_workspace(sizes),
            "norm_backward": lambda: lib.zo_block_norm_backward_workspace(block.NormArgs(T, D, 1, 0, 0, 0, 1e-5)),
            "conv_backward": lambda: lib.zo_conv_backward_workspace(block.ConvArgs(R, T, D, 4, 1, 0, 1))}[what]()
    assert need > 0
    ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
    want, got = run(None), run(ws[:need])
    for a, b in zip(got, want):
        assert torch.equal(a, b) and not torch.isnan(a).any()
    assert (ws[need:] == 255).all()
