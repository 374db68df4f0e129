"""The 64-bit references of the state-space block's operators: their gradient formulas
against central differences of their forwards, on the CPU."""
import pytest
import torch

from tests import block_reference as ref

F64 = torch.float64
H = 1e-6


def directional(f, tensors, weights):
    """Central difference of sum(f() * weights) along a random direction of each tensor, and the
    directions."""
    out = {}
    for name, t in tensors.items():
        v = torch.randn(t.shape, dtype=F64)
        keep = t.clone()
        vals = []
        for s in (H, -H):
            t.copy_(keep + s * v)
            vals.append(sum((a * w).sum() for a, w in zip(f(), weights)))
        t.copy_(keep)
        out[name] = ((vals[0] - vals[1]) / (2 * H), v)
    return out


def agree(diffs, grads):
    # a central difference with h = 1e-6 in 64 bits: h^2 times third derivatives of order 1..100
    # (1e-10) and 1e-16 / h times the value's size (1e-9)
    for name, (want, v) in diffs.items():
        got = (grads[name] * v).sum()
        assert abs(got - want) < 1e-6 * (1 + abs(want)), name


@pytest.mark.parametrize("act,ragged", [(True, True), (False, False)])
def test_conv_formula(act, ragged):
    torch.manual_seed(1)
    R, T, D, K, S = 4, 6, 3, 4, 2
    x, w, b = torch.randn(R, T, D, dtype=F64), torch.randn(S, K, D, dtype=F64), torch.randn(S, D, dtype=F64)
    st, dout, dst = torch.randn(R, K - 1, D, dtype=F64), torch.randn(R, T, D, dtype=F64), torch.randn(R, K - 1, D, dtype=F64)
    n = torch.tensor([6, 0, 1, 4]) if ragged else None

    def f():
        return ref.conv(x, w, b, act, n, st)[:2]
    dx, dw, db, ds = ref.conv_backward(x, w, dout, b, act, n, st, dst)
    on = ref.valid(n, R, T, "cpu")
    assert torch.all(torch.where(on, 0.0, dx) == 0)
    agree(directional(f, {"x": x, "w": w, "b": b, "s": st}, (dout, dst)),
          {"x": dx, "w": dw, "b": db, "s": ds})


@pytest.mark.parametrize("gate,softplus,ragged", [(True, True, True), (False, False, False)])
def test_scan_formula(gate, softplus, ragged):
    torch.manual_seed(2)
    R, T, D, G, N, S = 4, 7, 6, 2, 3, 2
    u, dl, z = (torch.randn(R, T, D, dtype=F64) for _ in range(3))
    B, C = (torch.randn(R, T, G, N, dtype=F64) for _ in range(2))
    A = -torch.rand(S, D, N, dtype=F64) - 0.2
    skip, bias = torch.randn(S, D, dtype=F64), torch.randn(S, D, dtype=F64)
    st, dst, dout = torch.randn(R, D, N, dtype=F64), torch.randn(R, D, N, dtype=F64), torch.randn(R, T, D, dtype=F64)
    n = torch.tensor([7, 0, 1, 5]) if ragged else None
    z = z if gate else None

    def f():
        return ref.scan(u, dl, A, B, C, skip, z, bias, softplus, n, st)[:2]
    g = ref.scan_backward(u, dl, A, B, C, dout, skip, z, bias, softplus, n, st, dst)
    names = {"du": u, "ddelta": dl, "dA": A, "dB": B, "dC": C, "dskip": skip, "ddelta_bias": bias, "dstate_in": st}
    if gate:
        names["dz"] = z
    agree(directional(f, names, (dout, dst)), g)


@pytest.mark.parametrize("gate_first", [False, True])
@pytest.mark.parametrize("without", ["", "w_post", "gate", "scale"])
def test_norm_formula(gate_first, without):
    if gate_first and without == "gate":
        pytest.skip("no gate to put first")
    torch.manual_seed(3)
    R, D, S = 4, 5, 2
    p = {"x": torch.randn(R, D, dtype=F64), "o": torch.randn(R, D, dtype=F64), "gate": torch.randn(R, D, dtype=F64)}
    p |= {k: torch.randn(S, D, dtype=F64) for k in ("w_post", "scale", "w_pre")}
    p.pop(without, None)
    x = p.pop("x")
    dxo, dn = torch.randn(R, D, dtype=F64), torch.randn(R, D, dtype=F64)

    def f():
        return ref.norm(x, eps=1e-3, gate_first=gate_first, **p)
    g = ref.norm_backward(f()[0], dn, dxo, eps=1e-3, gate_first=gate_first, **p)
    agree(directional(f, {"dx": x, **{"d" + k: v for k, v in p.items()}}, (dxo, dn)), g)
