"""Cases and plain forms of the linear-recurrence and block-norm operators.

The operators: ``linrec_solve`` / ``linrec_adjoint`` / ``linrec_step`` (the
gated linear recurrence, its adjoint and its single decode step) and
``block_norm`` / ``block_norm_adjoint`` (the norms around a block fused with
its gate and residual scale).  Each case runs one call of one of them.

``run`` computes a case with elementary torch operations in 32 bits where
``own`` is false, and with the library's entry points where it is true.
``exact`` computes the same from the definitions in 64 bits: the recurrence
step by step, gradients by automatic differentiation.
"""
import math

import torch

own = False

LIN_GRU, LIN_DECAY = "lin_gru", "lin_decay"
GATES = {LIN_GRU: 2, LIN_DECAY: 3}
KAPPA = 8.0
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
MAX_ELEMENTS = 1 << 27          # B * T * D of the largest listed recurrence


# ------------------------------------------------------------------ cases --
def listed():
    def rec(name, op, cell, B, T, D, dtype, docs=0, fused=False):
        return {"name": name, "op": op, "cell": cell, "B": B, "T": T, "D": D, "dtype": dtype,
                "docs": docs, "fused": fused}

    def norm(name, op, N, D, gate, post, res, scale, pre, dtype="bf16"):
        return {"name": name, "op": op, "N": N, "D": D, "gate": gate, "post": post, "res": res,
                "scale": scale, "pre": pre, "dtype": dtype}

    return [
        # one request's next token: latency
        rec("step_gru_b1", "step", LIN_GRU, 1, 1, 1024, "bf16"),
        # a full serving batch, u a part of a projection that also holds the gate
        rec("step_decay_b256", "step", LIN_DECAY, 256, 1, 4096, "bf16", fused=True),
        # a training layer at the default benchmark's shape
        rec("solve_gru_b8_t4096", "solve", LIN_GRU, 8, 4096, 1024, "bf16"),
        # one very long sequence in fp32
        rec("solve_decay_t65536", "solve", LIN_DECAY, 1, 65536, 2048, "f32"),
        # packed documents of uneven lengths, odd sizes, a strided u
        rec("solve_decay_docs", "solve", LIN_DECAY, 3, 1531, 1000, "bf16", docs=200, fused=True),
        # the training layer's backward pass
        rec("adjoint_gru_b8_t4096", "adjoint", LIN_GRU, 8, 4096, 1024, "bf16"),
        # wide channels and packed documents, backward
        rec("adjoint_decay_docs", "adjoint", LIN_DECAY, 4, 2048, 4096, "bf16", docs=512),
        # the pre-norm of one token in decoding
        norm("norm_token", "norm", 1, 4096, "", False, "bf16", False, True),
        # norm of the states, gate, scaled residual and the next pre-norm, whole batch
        norm("norm_block_n32768", "norm", 32768, 1024, "silu", True, "bf16", True, True),
        # gated output norm only, odd sizes
        norm("norm_gated_ragged", "norm", 4593, 1000, "sigmoid", True, "", False, False),
        # backward of the whole chain
        norm("norm_adjoint_n8192", "norm_adjoint", 8192, 4096, "silu", True, "bf16", True, True),
        # backward of a residual pre-norm, odd sizes, fp32 residual stream
        norm("norm_adjoint_pre", "norm_adjoint", 4593, 1000, "", False, "f32", False, True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "solve", "solve", "adjoint", "adjoint", "norm", "norm_adjoint"])
    D = 8 * _log_uniform(rng, 1, 512)
    if op in ("norm", "norm_adjoint"):
        post = rng.random() < 0.6
        return {"op": op, "N": _log_uniform(rng, 1, min(32768, (1 << 25) // D)), "D": D,
                "gate": rng.choice(["", "silu", "sigmoid"]), "post": post,
                "res": rng.choice(["", "bf16", "f32"]), "scale": rng.random() < 0.5,
                "pre": not post or rng.random() < 0.6, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op == "step":
        B, T = _log_uniform(rng, 1, 512), 1
    else:
        B = _log_uniform(rng, 1, 16)
        T = _log_uniform(rng, 1, min(65536, (MAX_ELEMENTS >> 2) // (B * D)))
    return {"op": op, "cell": rng.choice([LIN_GRU, LIN_DECAY]), "B": B, "T": T, "D": D,
            "dtype": rng.choice(["bf16", "bf16", "f32"]),
            "docs": rng.choice([0, 0, 16, 300]) if op != "step" else 0,
            "fused": rng.random() < 0.4}


def work(case):
    D = case["D"]
    e = BYTES[case["dtype"]]
    if "cell" in case:
        G = GATES[case["cell"]]
        n = case["B"] * case["T"] * D
        rows = 4 * case["B"] * D                     # h0, or dh0
        params = 4 * D * (G + (case["cell"] == LIN_DECAY))
        mask = case["B"] * case["T"] if case["docs"] else 0
        flops = n * (12 if case["cell"] == LIN_GRU else 25)
        if case["op"] == "adjoint":
            return {"bytes": 2 * G * n * e + 8 * n + 2 * rows + 2 * params + mask,
                    "flops": 2 * flops}
        return {"bytes": G * n * e + 4 * n + rows + params + mask, "flops": flops}
    n = case["N"] * D
    h = 4 if case["post"] else e                     # states are fp32, a projection's output is not
    g = e if case["gate"] else 0
    r = BYTES[case["res"]] if case["res"] else 0
    s = r or e
    x = e if case["pre"] else 0
    weights = 4 * D * (case["post"] + case["scale"] + case["pre"])
    if case["op"] == "norm":
        return {"bytes": n * (h + g + r + s + x) + weights, "flops": 15 * n}
    return {"bytes": n * (2 * h + 2 * g + 2 * r + s + x) + 2 * weights, "flops": 40 * n}


# ----------------------------------------------------------------- inputs --
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    D, dt = case["D"], TYPES[case["dtype"]]
    st = dict(case)
    if "cell" not in case:
        N = case["N"]
        st["h"] = randn(N, D) if case["post"] else randn(N, D).to(dt)
        st["g"] = randn(N, D).to(dt) if case["gate"] else None
        st["w_post"] = 1 + 0.1 * randn(D) if case["post"] else None
        st["res_in"] = (2 * randn(N, D)).to(TYPES[case["res"]]) if case["res"] else None
        st["scale_in"] = 0.5 + 0.1 * randn(D) if case["scale"] else None
        st["w_pre"] = 1 + 0.1 * randn(D) if case["pre"] else None
        st["s_dtype"] = TYPES[case["res"]] if case["res"] else dt
        if case["op"] == "norm_adjoint":
            st["ds"] = randn(N, D).to(st["s_dtype"])
            st["dx"] = randn(N, D).to(dt) if case["pre"] else None
        return st
    B, T, G = case["B"], case["T"], GATES[case["cell"]]
    if case["fused"]:       # one projection's output: G gate inputs and an output gate
        u = randn(B, T, (G + 1) * D).to(dt)[..., :G * D].unflatten(-1, (G, D))
    else:
        u = randn(B, T, G, D).to(dt)
    st["u"] = u
    st["bias"] = 0.1 * randn(G, D)
    st["h0"] = 0.5 * randn(B, D)
    st["lam"] = None
    if case["cell"] == LIN_DECAY:   # per-channel decays a = exp(-kappa softplus(lam)) of 0.9 to 0.999
        a = 0.9 + 0.099 * torch.rand(D, generator=gen, device="cuda")
        st["lam"] = torch.log(torch.expm1(-torch.log(a) / KAPPA))
    st["reset"] = None
    if case["docs"]:
        st["reset"] = torch.rand((B, T), generator=gen, device="cuda") < 1.0 / case["docs"]
    if case["op"] == "step":
        st["u"] = u[:, 0]
    if case["op"] == "adjoint":
        st["h"] = _plain_solve(st)
        st["dLdh"] = randn(B, T, D)
    return st


# ------------------------------------------------------------ plain forms --
def _gates(cell, u, lam, bias):
    """(a_t, b_t) of h_t = a_t h_{t-1} + b_t, and what the adjoint needs."""
    p = u.float() + bias
    if cell == LIN_GRU:
        z, a, c = torch.sigmoid(p[..., 0, :]), torch.sigmoid(-p[..., 0, :]), torch.tanh(p[..., 1, :])
        return a, z * c, (z, c)
    r, i, x = torch.sigmoid(p[..., 0, :]), torch.sigmoid(p[..., 1, :]), p[..., 2, :]
    y = 2 * KAPPA * torch.logaddexp(lam, torch.zeros_like(lam)) * r     # -2 log a
    beta = torch.sqrt(-torch.expm1(-y))
    return torch.exp(-0.5 * y), beta * i * x, (r, i, x, y, beta)


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from a zero state, by doubling."""
    n = 1
    while n < b.shape[1]:
        b = torch.cat([b[:, :n], torch.addcmul(b[:, n:], a[:, n:], b[:, :-n])], 1)
        a = torch.cat([a[:, :n], a[:, n:] * a[:, :-n]], 1)
        n *= 2
    return b


def _plain_solve(st):
    a, b, _ = _gates(st["cell"], st["u"], st["lam"], st["bias"])
    if st["reset"] is not None:
        a = a.masked_fill(st["reset"][..., None], 0.0)
    b[:, 0] += a[:, 0] * st["h0"]
    return _scan(a, b)


def _plain_step(st):
    a, b, _ = _gates(st["cell"], st["u"], st["lam"], st["bias"])
    return a * st["h0"] + b


def _plain_adjoint(st):
    u, h = st["u"], st["h"]
    a, _, saved = _gates(st["cell"], u, st["lam"], st["bias"])
    hp = torch.cat([st["h0"][:, None], h[:, :-1]], 1)
    if st["reset"] is not None:
        a = a.masked_fill(st["reset"][..., None], 0.0)
        hp = hp.masked_fill(st["reset"][..., None], 0.0)
    after = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    lam_t = _scan(after.flip(1), st["dLdh"].flip(1)).flip(1)
    out = {"dh0": a[:, 0] * lam_t[:, 0]}
    if st["cell"] == LIN_GRU:
        z, c = saved
        du = torch.stack([lam_t * (c - hp) * z * torch.sigmoid(-(u[..., 0, :].float() + st["bias"][0])),
                          lam_t * z * (1 - c * c)], 2)
    else:
        r, i, x, y, beta = saved
        keep = torch.exp(-0.5 * y)
        e = lam_t * 0.5 * y * (keep * keep * i * x / beta - keep * hp)   # r dL/dr
        one = u.float() + st["bias"]
        du = torch.stack([e * torch.sigmoid(-one[..., 0, :]),
                          lam_t * beta * x * i * torch.sigmoid(-one[..., 1, :]),
                          lam_t * beta * i], 2)
        sp = torch.logaddexp(st["lam"], torch.zeros_like(st["lam"]))
        out["dlam"] = e.sum((0, 1)) * torch.sigmoid(st["lam"]) / sp
    out["dbias"] = du.sum((0, 1))
    out["du"] = du.to(u.dtype)
    return out


def _act(name, g):
    """(act(g), act'(g))"""
    q = torch.sigmoid(g)
    if name == "sigmoid":
        return q, q * torch.sigmoid(-g)
    return g * q, q * (1 + g * torch.sigmoid(-g))


def _rstd(v):
    return torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)


def _plain_norm(st):
    y = st["h"].float()
    if st["w_post"] is not None:
        y = y * _rstd(y) * st["w_post"]
    if st["g"] is not None:
        y = y * _act(st["gate"], st["g"].float())[0]
    if st["scale_in"] is not None:
        y = y * st["scale_in"]
    s = y if st["res_in"] is None else st["res_in"].float() + y
    out = {"s": s.to(st["s_dtype"])}
    if st["w_pre"] is not None:
        out["x"] = (s * _rstd(s) * st["w_pre"]).to(TYPES[st["dtype"]])
    return out


def _plain_norm_adjoint(st):
    h = st["h"].float()
    n = h
    if st["w_post"] is not None:
        k = _rstd(h)
        hat = h * k
        n = hat * st["w_post"]
    if st["g"] is not None:
        act, dact = _act(st["gate"], st["g"].float())
        y = n * act
    else:
        y = n
    s = y if st["scale_in"] is None else y * st["scale_in"]
    if st["res_in"] is not None:
        s = st["res_in"].float() + s
    out, d = {}, st["ds"].float()
    if st["w_pre"] is not None:
        ks = _rstd(s)
        sh, dx = s * ks, st["dx"].float()
        out["dw_pre"] = (dx * sh).sum(0)
        dx = dx * st["w_pre"]
        d = d + ks * (dx - sh * (dx * sh).mean(-1, keepdim=True))
    if st["res_in"] is not None:
        out["dres"] = d.to(st["res_in"].dtype)
    if st["scale_in"] is not None:
        out["dscale"] = (d * y).sum(0)
        d = d * st["scale_in"]
    if st["g"] is not None:
        out["dgate"] = (d * n * dact).to(st["g"].dtype)
        d = d * act
    if st["w_post"] is not None:
        out["dw_post"] = (d * hat).sum(0)
        d = d * st["w_post"]
        d = k * (d - hat * (d * hat).mean(-1, keepdim=True))
    out["dh"] = d.to(st["h"].dtype)
    return out


PLAIN = {"solve": _plain_solve, "step": _plain_step, "adjoint": _plain_adjoint,
         "norm": _plain_norm, "norm_adjoint": _plain_norm_adjoint}


# -------------------------------------------------------- the entry points --
def _own(st):
    import nonlinear_rnn_paragru_b200 as pr
    op = st["op"]
    if op in ("norm", "norm_adjoint"):
        parts = dict(gate=st["g"], act=st["gate"] or "silu", w_post=st["w_post"], res=st["res_in"],
                     scale=st["scale_in"], w_pre=st["w_pre"], eps=EPS)
        if op == "norm":
            s, x = pr.block_norm(st["h"], s_dtype=st["s_dtype"], x_dtype=TYPES[st["dtype"]], **parts)
            return {"s": s} if x is None else {"s": s, "x": x}
        out = pr.block_norm_adjoint(st["h"], st["ds"], st["dx"], **parts)
        return {k: v for k, v in out.items() if v is not None}
    cell = pr.PARARNN_LIN_GRU if st["cell"] == LIN_GRU else pr.PARARNN_LIN_DECAY
    if op == "step":
        return pr.linrec_step(cell, st["u"], st["lam"], st["bias"], st["h0"], kappa=KAPPA)
    if op == "solve":
        return pr.linrec_solve(cell, st["u"], st["lam"], st["bias"], st["h0"], reset=st["reset"],
                               kappa=KAPPA)
    out = pr.linrec_adjoint(cell, st["u"], st["lam"], st["bias"], st["h0"], st["h"], st["dLdh"],
                            reset=st["reset"], kappa=KAPPA)
    return {k: v for k, v in out.items() if v is not None}


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ----------------------------------------------------------- the 64 bits --
def _exact_coefficients(st, u, lam, bias):
    pre = [u[..., k, :] + bias[k] for k in range(u.shape[-2])]
    if st["cell"] == LIN_GRU:
        z = 1 / (1 + torch.exp(-pre[0]))
        return 1 - z, z * torch.tanh(pre[1])
    loga = -KAPPA * torch.nn.functional.softplus(lam, threshold=1e9) / (1 + torch.exp(-pre[0]))
    return torch.exp(loga), torch.sqrt(-torch.expm1(2 * loga)) / (1 + torch.exp(-pre[1])) * pre[2]


def _exact_states(st, a, b, h0):
    hs, h = [], h0
    for t in range(b.shape[1]):
        if st["reset"] is not None:
            h = h * (~st["reset"][:, t, None])
        h = a[:, t] * h + b[:, t]
        hs.append(h)
    return torch.stack(hs, 1)


def _exact_adjoint(st, u, lam, bias, h0):
    """du_t = (dh_t/du_t)^T lambda_t with the given states h as the trajectory."""
    h, g = st["h"].double(), st["dLdh"].double()
    hp = torch.cat([h0[:, None], h[:, :-1]], 1)
    keep = torch.ones_like(hp[..., :1]) if st["reset"] is None else (~st["reset"])[..., None].double()
    with torch.no_grad():
        a = _exact_coefficients(st, u, lam, bias)[0] * keep
        lt, carry = torch.empty_like(g), torch.zeros_like(h0)
        for t in reversed(range(g.shape[1])):
            lt[:, t] = g[:, t] + carry
            carry = a[:, t] * lt[:, t]
    out = {"dh0": carry}
    del a
    leaves = [u, bias] + ([lam] if lam is not None else [])
    for v in leaves:
        v.requires_grad_(True)
    a, b = _exact_coefficients(st, u, lam, bias)
    loss = ((a * (hp * keep) + b) * lt).sum()
    grads = torch.autograd.grad(loss, leaves)
    out["du"], out["dbias"] = grads[0], grads[1]
    if lam is not None:
        out["dlam"] = grads[2]
    return {k: v.detach() for k, v in out.items()}


def _exact_norm(st, v):
    y = v["h"]
    D = y.shape[-1]
    if v["w_post"] is not None:
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / D + EPS) * v["w_post"]
    if v["g"] is not None:
        y = y / (1 + torch.exp(-v["g"])) * (v["g"] if st["gate"] == "silu" else 1)
    y = y * (1 if v["scale_in"] is None else v["scale_in"])
    s = y + (0 if v["res_in"] is None else v["res_in"])
    if v["w_pre"] is None:
        return {"s": s}
    return {"s": s, "x": s / torch.sqrt((s * s).sum(-1, keepdim=True) / D + EPS) * v["w_pre"]}


NAMES = {"h": "dh", "g": "dgate", "w_post": "dw_post", "res_in": "dres", "scale_in": "dscale",
         "w_pre": "dw_pre"}


def exact(case, seed):
    st = prepare(case, seed)
    wide = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v
            for k, v in st.items()}
    if "cell" in case:
        u, lam, bias, h0 = wide["u"], wide["lam"], wide["bias"], wide["h0"]
        if case["op"] == "adjoint":
            return _exact_adjoint(st, u, lam, bias, h0)
        a, b = _exact_coefficients(st, u, lam, bias)
        return a * h0 + b if case["op"] == "step" else _exact_states(st, a, b, h0)
    if case["op"] == "norm":
        return _exact_norm(st, wide)
    leaves = {k: wide[k].requires_grad_(True) for k in NAMES if wide[k] is not None}
    out = _exact_norm(st, wide)
    loss = (out["s"] * wide["ds"]).sum()
    if "x" in out:
        loss = loss + (out["x"] * wide["dx"]).sum()
    grads = torch.autograd.grad(loss, list(leaves.values()))
    return {NAMES[k]: g for k, g in zip(leaves, grads)}
