"""The selective state-space block's operators: measured cases and their plain forms.

Three operators, each in the forms that a program uses:

* conv  - the short causal convolution over time with its SiLU: prompts
          (padded rows of unequal lengths), training (forward and backward),
          single tokens (a window of the last inputs is carried).
* scan  - the selective scan h_t = exp(d_t A) h_{t-1} + d_t B_t u_t,
          y_t = C_t h_t + skip u_t, gated by silu(z_t), with
          d_t = softplus(delta_t + bias): prompts, training, single tokens.
* norm  - the join of two blocks: a norm after the block with its gate and
          residual scale, the residual addition, and the next block's norm.

Parameters are fp32 and may come as several sets (one per perturbed copy of a
model); the rows are then divided evenly among the sets, in order.  Everything
here computes in 32 bits and rounds once where `own` is false; `exact` computes
in 64 bits, step by step.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---- cases --------------------------------------------------------------------

def listed():
    scan = {"op": "scan", "groups": 1, "n": 16, "sets": 1, "ragged": False, "gate": True, "dtype": "bf16"}
    conv = {"op": "conv", "k": 4, "sets": 1, "ragged": False, "dtype": "bf16"}
    norm = {"op": "norm", "form": "forward", "sets": 1, "dtype": "bf16", "residual": "f32"}
    return [
        # one user's next token: nothing but latency
        {**scan, "name": "scan_step_one", "form": "step", "rows": 1, "seq": 1, "d": 2048},
        # the next token of a full serving batch: the states' traffic
        {**scan, "name": "scan_step_batch", "form": "step", "rows": 512, "seq": 1, "d": 4096},
        # probe losses: many short rows (char-LM length 10), 8 perturbed parameter sets
        {**scan, "name": "scan_probes", "form": "prompt", "rows": 4096, "seq": 10, "d": 1024, "sets": 8},
        # one long prompt: few rows, so time itself has to be divided
        {**scan, "name": "scan_prompt_long", "form": "prompt", "rows": 1, "seq": 16384, "d": 2048},
        # a training step of the scan: forward and all gradients
        {**scan, "name": "scan_train", "form": "train", "rows": 4, "seq": 2048, "d": 2048},
        # odd sizes throughout: unequal lengths, four groups, 24 states, fp32
        {**scan, "name": "scan_train_ragged", "form": "train", "rows": 6, "seq": 777, "d": 520, "groups": 4, "n": 24, "ragged": True, "dtype": "f32"},
        # a batch of prompts through the convolution: memory traffic
        {**conv, "name": "conv_prompt", "form": "prompt", "rows": 8, "seq": 2048, "d": 4096},
        # a training step of the convolution on odd sizes and unequal lengths
        {**conv, "name": "conv_train_ragged", "form": "train", "rows": 5, "seq": 1999, "d": 1344, "k": 3, "ragged": True, "dtype": "f16"},
        # the next token of a serving batch
        {**conv, "name": "conv_step", "form": "step", "rows": 64, "seq": 1, "d": 4096},
        # the join of two blocks over a batch of prompts
        {**norm, "name": "norm_join", "rows": 16384, "d": 4096},
        # the same for eight single tokens
        {**norm, "name": "norm_join_small", "rows": 8, "d": 1024},
        # forward and all gradients, four parameter sets
        {**norm, "name": "norm_train", "form": "train", "rows": 8192, "d": 2048, "sets": 4},
    ]


def draw(rng):
    def span(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["scan", "scan", "scan", "conv", "conv", "norm", "norm"])
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"])}
    if op == "norm":
        case["form"] = rng.choice(["forward", "train"])
        case["d"] = span(33, 8192)
        case["sets"] = rng.choice([1, 1, 2, 5])
        most = 33_000_000 if case["form"] == "forward" else 16_000_000
        case["rows"] = case["sets"] * span(1, max(2, min(16384, most // case["d"]) // case["sets"]))
        case["residual"] = rng.choice(["f32", case["dtype"]])
        return case
    case["form"] = rng.choice(["step", "prompt", "train"])
    case["sets"] = rng.choice([1, 1, 1, 2, 4])
    case["ragged"] = case["form"] != "step" and rng.random() < 0.5
    if op == "conv":
        case["k"] = rng.choice([2, 3, 4, 4, 5, 8])
        case["d"] = span(17, 8192)
        most = 33_000_000 if case["form"] == "prompt" else 13_000_000
    else:
        case["groups"] = rng.choice([1, 1, 2, 4])
        case["d"] = case["groups"] * span(8, 4096 // case["groups"])
        case["n"] = rng.choice([4, 7, 8, 16, 16, 16, 24, 32, 64])
        case["gate"] = rng.random() < 0.7
        most = {"prompt": min(480_000_000 // case["n"], 33_000_000), "train": min(200_000_000 // case["n"], 16_000_000), "step": 30_000_000 // case["n"]}[case["form"]]
    if case["form"] == "step":
        case["seq"] = 1
        case["rows"] = case["sets"] * span(1, max(1, min(512, most // case["d"]) // case["sets"]))
    else:
        case["seq"] = span(1, 8192)
        case["rows"] = case["sets"] * span(1, max(1, min(512, most // (case["d"] * case["seq"])) // case["sets"]))
        case["seq"] = max(1, min(case["seq"], most // (case["d"] * case["rows"])))
    return case


# ---- inputs --------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.float32, scale=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale + mean).to(dtype)

    dt, R, D, S = DT[case["dtype"]], case["rows"], case["d"], case["sets"]
    s = {"case": dict(case)}
    if case["op"] == "norm":
        xt = DT[case["residual"]]
        s["x"] = normal(R, D, dtype=xt, scale=2.0)
        s["o"] = normal(R, D, dtype=dt, scale=0.5)
        s["gate"] = normal(R, D, dtype=dt)
        s["w_post"] = normal(S, D, scale=0.1, mean=1.0)
        s["scale"] = normal(S, D, scale=0.02, mean=0.1)
        s["w_pre"] = normal(S, D, scale=0.1, mean=1.0)
        s["x_out"], s["n_out"] = torch.empty_like(s["x"]), torch.empty_like(s["o"])
        if case["form"] == "train":
            s["dn"], s["dx_out"] = normal(R, D, dtype=dt), normal(R, D, dtype=xt)
            s["dx"], s["do"], s["dgate"] = torch.empty_like(s["x"]), torch.empty_like(s["o"]), torch.empty_like(s["o"])
            s["dw_post"], s["dscale"], s["dw_pre"] = (torch.empty(S, D, device="cuda") for _ in range(3))
        return s

    T = case["seq"]
    step, train = case["form"] == "step", case["form"] == "train"
    time = () if step else (T,)
    s["lengths"] = None
    if case["ragged"]:
        n = torch.randint(0, T + 1, (R,), generator=g, device="cuda", dtype=torch.int32)
        n[0] = T
        s["lengths"] = n
    if case["op"] == "conv":
        K = case["k"]
        s["x"] = normal(R, *time, D, dtype=dt)
        s["weight"], s["bias"] = normal(S, K, D, scale=K ** -0.5), normal(S, D, scale=0.1)
        s["out"] = torch.empty_like(s["x"])
        s["state"] = None if train else normal(R, K - 1, D, dtype=dt)
        s["state_out"] = None if train else torch.empty_like(s["state"])
        if train:
            s["dout"] = normal(R, T, D, dtype=dt)
            s["dx"] = torch.empty_like(s["x"])
            s["dweight"], s["dbias"] = torch.empty(S, K, D, device="cuda"), torch.empty(S, D, device="cuda")
        return s

    N, G = case["n"], case["groups"]
    s["u"] = normal(R, *time, D, dtype=dt)
    s["delta"] = normal(R, *time, D, dtype=dt, scale=0.5)
    s["z"] = normal(R, *time, D, dtype=dt) if case["gate"] else None
    s["B"], s["C"] = (normal(R, *time, G, N, dtype=dt) for _ in range(2))
    # decay rates -1..-N and steps of 0.001..0.1, the usual start, each copy perturbed a little
    s["A"] = -torch.arange(1, N + 1, device="cuda").float().expand(S, D, N) * (1 + normal(S, D, N, scale=0.01))
    step0 = torch.exp(torch.rand(S, D, generator=g, device="cuda") * math.log(100.0) + math.log(0.001))
    s["delta_bias"] = torch.log(torch.expm1(step0))
    s["skip"] = normal(S, D, scale=0.1, mean=1.0)
    s["out"] = torch.empty_like(s["u"])
    s["state"] = None if train else normal(R, D, N)
    s["state_out"] = None if train else torch.empty(R, D, N, device="cuda")
    if train:
        s["dout"] = normal(R, T, D, dtype=dt)
        s["du"], s["ddelta"] = torch.empty_like(s["u"]), torch.empty_like(s["u"])
        s["dz"] = torch.empty_like(s["u"]) if case["gate"] else None
        s["dB"], s["dC"] = torch.empty_like(s["B"]), torch.empty_like(s["C"])
        s["dA"] = torch.empty(S, D, N, device="cuda")
        s["dskip"], s["ddelta_bias"] = torch.empty(S, D, device="cuda"), torch.empty(S, D, device="cuda")
    return s


# ---- one pass --------------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        return {"norm": _own_norm, "conv": _own_conv, "scan": _own_scan}[case["op"]](state, case["form"])
    return {"norm": _norm, "conv": _conv, "scan": _scan}[case["op"]](state, case["form"])


def _own_norm(s, form):
    import zero_order_recurrent_b200 as zo
    p = {"o": s["o"], "gate": s["gate"], "w_post": s["w_post"], "scale": s["scale"], "w_pre": s["w_pre"], "eps": 1e-5}
    zo.zo_block_norm(s["x"], x_out=s["x_out"], n_out=s["n_out"], **p)
    if form != "train":
        return [s["x_out"], s["n_out"]]
    zo.zo_block_norm_backward(s["x_out"], dn=s["dn"], dx_out=s["dx_out"], dx=s["dx"], do=s["do"], dgate=s["dgate"],
                              dw_post=s["dw_post"], dscale=s["dscale"], dw_pre=s["dw_pre"], **p)
    return [s[k] for k in ("x_out", "n_out", "dx", "do", "dgate", "dw_post", "dscale", "dw_pre")]


def _own_conv(s, form):
    import zero_order_recurrent_b200 as zo
    if form == "step":
        zo.zo_conv_step(s["x"], s["weight"], s["state"], s["out"], bias=s["bias"], state_out=s["state_out"])
        return [s["out"], s["state_out"]]
    zo.zo_conv(s["x"], s["weight"], s["out"], bias=s["bias"], lengths=s["lengths"], state_in=s["state"], state_out=s["state_out"])
    if form == "prompt":
        return [s["out"], s["state_out"]]
    zo.zo_conv_backward(s["x"], s["weight"], s["dout"], s["dx"], s["dweight"], bias=s["bias"], dbias=s["dbias"], lengths=s["lengths"])
    return [s["out"], s["dx"], s["dweight"], s["dbias"]]


def _own_scan(s, form):
    import zero_order_recurrent_b200 as zo
    p = {"skip": s["skip"], "z": s["z"], "delta_bias": s["delta_bias"], "softplus": True}
    if form == "step":
        zo.zo_scan_step(s["u"], s["delta"], s["A"], s["B"], s["C"], s["state"], s["out"], state_out=s["state_out"], **p)
        return [s["out"], s["state_out"]]
    p["lengths"] = s["lengths"]
    if form == "prompt":
        zo.zo_scan(s["u"], s["delta"], s["A"], s["B"], s["C"], s["out"], state_in=s["state"], state_out=s["state_out"], **p)
        return [s["out"], s["state_out"]]
    kept = torch.empty(zo.zo_scan_checkpoint_shape(s["u"].shape, s["A"].shape[-1]), device=s["u"].device)
    zo.zo_scan(s["u"], s["delta"], s["A"], s["B"], s["C"], s["out"], checkpoints=kept, **p)
    zo.zo_scan_backward(s["u"], s["delta"], s["A"], s["B"], s["C"], s["dout"], kept, s["du"], s["ddelta"], s["dA"], s["dB"], s["dC"],
                        dskip=s["dskip"], dz=s["dz"], ddelta_bias=s["ddelta_bias"], **p)
    return [s[k] for k in ("out", "du", "ddelta", "dA", "dB", "dC", "dskip", "dz", "ddelta_bias") if s[k] is not None]


# ---- plain forms: 32 bits, rounded once at the end -----------------------------

def _silu(x):
    return x / (1 + torch.exp(-x))


def _dsilu(x):
    q = 1 / (1 + torch.exp(-x))
    return q * (1 + x * (1 - q))


def _rows(p, rows):
    """Parameters [sets, ...] as [rows, ...]."""
    return p.repeat_interleave(rows // p.shape[0], 0)


def _by_set(v, sets):
    """Sums of [rows, ...] over the rows of each set."""
    return v.reshape(sets, -1, *v.shape[1:]).sum(1)


def _valid(lengths, rows, T):
    t = torch.arange(T, device="cuda")
    return torch.ones(rows, T, dtype=torch.bool, device="cuda") if lengths is None else t < lengths[:, None]


def _norm(s, form):
    S, eps = s["case"]["sets"], 1e-5
    R, D = s["x"].shape
    x, o, gate = s["x"].float(), s["o"].float(), s["gate"].float()
    wp, sc, wn = (s[k].repeat_interleave(R // S, 0) for k in ("w_post", "scale", "w_pre"))
    ro = torch.rsqrt((o * o).mean(-1, keepdim=True) + eps)
    act = _silu(gate)
    xo = x + sc * (o * ro * wp * act)
    n = xo * torch.rsqrt((xo * xo).mean(-1, keepdim=True) + eps) * wn
    out = [xo.to(s["x"].dtype), n.to(s["o"].dtype)]
    if form != "train":
        return out
    y, dn = out[0].float(), s["dn"].float()       # the backward pass starts from the stored residual
    ry = torch.rsqrt((y * y).mean(-1, keepdim=True) + eps)
    dh = dn * wn
    dx = s["dx_out"].float() + ry * (dh - y * ry * ry * (dh * y).mean(-1, keepdim=True))
    dp = dx * sc
    dv = dp * act * wp
    do = ro * (dv - o * ro * ro * (dv * o).mean(-1, keepdim=True))
    dgate = dp * o * ro * wp * _dsilu(gate)
    return out + [dx.to(s["x"].dtype), do.to(s["o"].dtype), dgate.to(s["o"].dtype), _by_set(dp * act * o * ro, S),
                  _by_set(dx * o * ro * wp * act, S), _by_set(dn * y * ry, S)]


def _conv(s, form):
    S, K, R, dt = s["case"]["sets"], s["case"]["k"], s["x"].shape[0], s["x"].dtype
    w, b = _rows(s["weight"], R), _rows(s["bias"], R)[:, None]
    x = s["x"].float() if form != "step" else s["x"].float()[:, None]
    T = x.shape[1]
    on = _valid(s["lengths"], R, T)[..., None]
    x = torch.where(on, x, 0.0)
    before = torch.zeros(R, K - 1, x.shape[2], device="cuda") if s["state"] is None else s["state"].float()
    xp = torch.cat([before, x], 1)
    win = xp.unfold(1, K, 1)                                    # [R, T, D, K]
    pre = (win * w.transpose(1, 2)[:, None]).sum(-1) + b
    out = torch.where(on, _silu(pre), 0.0).to(dt)
    if form == "step":
        return [out[:, 0], xp[:, 1:].to(dt)]
    if form == "prompt":
        n = torch.full((R,), T, device="cuda") if s["lengths"] is None else s["lengths"].long()
        at = n[:, None] + torch.arange(K - 1, device="cuda")
        return [out, xp.gather(1, at[..., None].expand(-1, -1, x.shape[2])).to(dt)]
    d = torch.where(on, s["dout"].float() * _dsilu(pre), 0.0)
    dw = _by_set((win * d[..., None]).sum(1).transpose(1, 2), S)
    tail = torch.cat([d, torch.zeros(R, K - 1, x.shape[2], device="cuda")], 1).unfold(1, K, 1)
    dx = (tail * w.flip(1).transpose(1, 2)[:, None]).sum(-1)
    return [out, torch.where(on, dx, 0.0).to(dt), dw, _by_set(d.sum(1), S)]


def _recur(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1, in log2(T) doublings."""
    s = 1
    while s < a.shape[1]:
        b = torch.cat([b[:, :s], b[:, s:] + a[:, s:] * b[:, :-s]], 1)
        a = torch.cat([a[:, :s], a[:, s:] * a[:, :-s]], 1)
        s *= 2
    return b


def _scan(s, form):
    S, G, R, D, dt = s["case"]["sets"], s["case"]["groups"], s["u"].shape[0], s["u"].shape[-1], s["u"].dtype
    step = form == "step"
    u, delta, B, C = (s[k].float()[:, None] if step else s[k].float() for k in ("u", "delta", "B", "C"))
    B, C = B.repeat_interleave(D // G, 2), C.repeat_interleave(D // G, 2)      # [R, T, D, N]
    A, skip, bias = _rows(s["A"], R)[:, None], _rows(s["skip"], R)[:, None], _rows(s["delta_bias"], R)[:, None]
    T = u.shape[1]
    on = _valid(s["lengths"], R, T)[..., None]
    raw = delta + bias
    d = torch.where(on, torch.where(raw > 20, raw, torch.log1p(torch.exp(raw.clamp(max=20)))), 0.0)
    a = torch.exp(d[..., None] * A)
    b = (d * u)[..., None] * B
    if s["state"] is not None:
        b = torch.cat([b[:, :1] + a[:, :1] * s["state"][:, None], b[:, 1:]], 1)
    h = _recur(a, b)
    y = (h * C).sum(-1) + skip * u
    z = None if s["z"] is None else s["z"].float()[:, None] if step else s["z"].float()
    out = torch.where(on, y if z is None else y * _silu(z), 0.0).to(dt)
    if step:
        return [out[:, 0], h[:, 0]]
    if form == "prompt":
        return [out, h[:, -1]]
    dout = torch.where(on, s["dout"].float(), 0.0)
    dy = dout if z is None else dout * _silu(z)
    dz = None if z is None else dout * y * _dsilu(z)
    nxt = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    gr = _recur(nxt.flip(1), (C * dy[..., None]).flip(1)).flip(1)
    ah = a * torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    gB = (gr * B).sum(-1)
    draw_ = ((gr * ah * A).sum(-1) + gB * u) * (1 / (1 + torch.exp(-raw)))
    draw_ = torch.where(on, draw_, 0.0)
    du = gB * d + skip * dy
    dB = (gr * (d * u)[..., None]).reshape(R, T, G, D // G, -1).sum(3)
    dC = (h * dy[..., None]).reshape(R, T, G, D // G, -1).sum(3)
    dA = _by_set((gr * ah * d[..., None]).sum(1), S)
    got = [out, du.to(dt), draw_.to(dt), dA, dB.to(dt), dC.to(dt), _by_set((dy * u).sum(1), S), None if dz is None else dz.to(dt), _by_set(draw_.sum(1), S)]
    return [v for v in got if v is not None]


# ---- work --------------------------------------------------------------------

def work(case):
    e = torch.finfo(DT[case["dtype"]]).bits // 8
    R, D, S, train = case["rows"], case["d"], case["sets"], case["form"] == "train"
    if case["op"] == "norm":
        x = torch.finfo(DT[case["residual"]]).bits // 8
        m = R * D
        if train:
            return {"bytes": m * (2 * x + 3 * e) + m * (2 * x + 4 * e) + 24 * S * D, "flops": 50.0 * m}
        return {"bytes": m * (2 * x + 3 * e) + 12 * S * D, "flops": 16.0 * m}
    m = R * case["seq"] * D
    if case["op"] == "conv":
        K = case["k"]
        if train:
            return {"bytes": 4 * m * e + 8 * S * D * (K + 1), "flops": m * (6.0 * K + 20)}
        return {"bytes": 2 * m * e + 2 * R * (K - 1) * D * e + 4 * S * D * (K + 1), "flops": m * (2.0 * K + 6)}
    N, G, z = case["n"], case["groups"], 1 if case["gate"] else 0
    bc = 2 * R * case["seq"] * G * N * e
    if train:  # in: u, delta, z, dout; out: out, du, ddelta, dz
        return {"bytes": m * e * (6 + 2 * z) + 2 * bc + 8 * S * D * (N + 2), "flops": m * (20.0 * N + 40)}
    return {"bytes": m * e * (3 + z) + bc + 8 * R * D * N + 4 * S * D * (N + 2), "flops": m * (7.0 * N + 20)}


# ---- 64 bits, step by step -----------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad() if case["op"] == "scan" else torch.enable_grad():
        return {"norm": _exact_norm, "conv": _exact_conv, "scan": _exact_scan}[case["op"]](s, case)


def _each(p, rows):
    """The parameters that each row uses, in 64 bits."""
    return p.double()[torch.arange(rows, device="cuda") // (rows // p.shape[0])]


def _exact_norm(s, case):
    R = case["rows"]
    q = {k: s[k].double().requires_grad_() for k in ("x", "o", "gate", "w_post", "scale", "w_pre")}
    wp, sc, wn = (_each(q[k], R) for k in ("w_post", "scale", "w_pre"))

    def unit(v):
        return v / torch.sqrt(v.pow(2).mean(1, keepdim=True) + 1e-5)

    add = sc * unit(q["o"]) * wp * q["gate"] * torch.sigmoid(q["gate"])
    xo = q["x"] + add
    n = unit(xo) * wn
    if case["form"] != "train":
        return [xo.detach(), n.detach()]
    # gradients at the residual as it is stored
    stored = (xo.detach().to(s["x"].dtype).double() - add.detach())
    xo2 = stored + add + (q["x"] - q["x"].detach())
    loss = (unit(xo2) * wn * s["dn"].double()).sum() + (xo2 * s["dx_out"].double()).sum()
    g = torch.autograd.grad(loss, [q[k] for k in ("x", "o", "gate", "w_post", "scale", "w_pre")])
    return [xo.detach(), n.detach(), *g]


def _exact_conv(s, case):
    R, K, T = case["rows"], case["k"], case["seq"]
    x = s["x"].double() if case["form"] != "step" else s["x"].double().unsqueeze(1)
    x.requires_grad_()
    w, b = s["weight"].double().requires_grad_(), s["bias"].double().requires_grad_()
    wr, br = _each(w, R), _each(b, R)
    past = torch.zeros(R, K - 1, case["d"], device="cuda", dtype=torch.float64) if s["state"] is None else s["state"].double()
    xs = torch.cat([past, x], 1)
    n = torch.full((R,), T, device="cuda") if s["lengths"] is None else s["lengths"].long()
    acc = br[:, None].expand(R, T, case["d"])
    for k in range(K):
        acc = acc + wr[:, k, None] * xs[:, k:k + T]
    out = acc * torch.sigmoid(acc)
    out = out * (torch.arange(T, device="cuda")[None] < n[:, None]).unsqueeze(-1)
    if case["form"] != "train":
        last = torch.stack([xs[r, int(m):int(m) + K - 1] for r, m in enumerate(n.tolist())])
        return [out.detach()[:, 0] if case["form"] == "step" else out.detach(), last.detach()]
    dx, dw, db = torch.autograd.grad((out * s["dout"].double()).sum(), [x, w, b])
    return [out.detach(), dx, dw, db]


def _exact_scan(s, case):
    R, T, D, N, G, S = (case[k] for k in ("rows", "seq", "d", "n", "groups", "sets"))
    step, train = case["form"] == "step", case["form"] == "train"
    if R * D * N * T > 600_000_000 and train:
        return None
    A, skip, bias = _each(s["A"], R), _each(s["skip"], R), _each(s["delta_bias"], R)
    of = torch.arange(D, device="cuda") // (D // G)
    n = torch.full((R,), T, device="cuda") if s["lengths"] is None else s["lengths"].long()

    def at(k, t):
        return s[k].double() if step else s[k][:, t].double()

    def steps(t):
        raw = at("delta", t) + bias
        d = torch.logaddexp(raw, torch.zeros_like(raw)) * (t < n)[:, None]
        return raw, d, torch.exp(d[..., None] * A), at("B", t)[:, of], at("C", t)[:, of]

    h = torch.zeros(R, D, N, device="cuda", dtype=torch.float64) if s["state"] is None else s["state"].double()
    out = torch.zeros(R, T, D, device="cuda", dtype=torch.float64)
    kept = [h]
    for t in range(T):
        raw, d, a, B, C = steps(t)
        h = a * h + (d * at("u", t))[..., None] * B
        y = torch.einsum("rdn,rdn->rd", h, C) + skip * at("u", t)
        if s["z"] is not None:
            y = y * at("z", t) * torch.sigmoid(at("z", t))
        out[:, t] = y * (t < n)[:, None]
        if train:
            kept.append(h)
    if not train:
        return [out[:, 0] if step else out, h]
    new = {k: torch.zeros_like(s[k], dtype=torch.float64) for k in ("du", "ddelta", "dB", "dC", "u")}
    dz = torch.zeros_like(new["u"])
    dA, dskip, dbias = torch.zeros(R, D, N, device="cuda", dtype=torch.float64), 0, 0
    carry = torch.zeros_like(dA)
    for t in reversed(range(T)):
        raw, d, a, B, C = steps(t)
        u, dy = at("u", t), at("dout", t) * (t < n)[:, None]
        if s["z"] is not None:
            zt = at("z", t)
            q = torch.sigmoid(zt)
            y = (kept[t + 1] * C).sum(-1) + skip * u
            dz[:, t] = dy * y * (q + zt * q * (1 - q))
            dy = dy * zt * q
        carry = carry + C * dy[..., None]
        new["dC"][:, t] = (kept[t + 1] * dy[..., None]).view(R, G, D // G, N).sum(2)
        new["dB"][:, t] = (carry * (d * u)[..., None]).view(R, G, D // G, N).sum(2)
        through = carry * a * kept[t]
        gb = (carry * B).sum(-1)
        dd = ((through * A).sum(-1) + gb * u) * torch.sigmoid(raw) * (t < n)[:, None]
        new["ddelta"][:, t] = dd
        new["du"][:, t] = gb * d + skip * dy
        dA = dA + through * d[..., None]
        dskip, dbias = dskip + dy * u, dbias + dd
        carry = carry * a

    def total(v):
        return torch.stack([c.sum(0) for c in v.chunk(S, 0)])

    got = [out, new["du"], new["ddelta"], total(dA), new["dB"], new["dC"], total(dskip)]
    return got + ([dz] if s["z"] is not None else []) + [total(dbias)]
