"""fp64 restatement of the gated linear recurrence and the block norm, in plain
numpy: the recurrence step by step, the adjoints from the formulas.

TEST INFRASTRUCTURE ONLY; shares no code with the CUDA path.  Besides each
result the functions return a *magnitude*: the same expression with every term
replaced by its absolute value.  An fp32 evaluation of k roundings is off by at
most about k 2^-24 times that, cancellation or not, so the tests' tolerances
are multiples of it.

Pins (tests/test_layer_cpu.py): torch autograd in float64 and central
differences for both adjoints; ParaGRU's own oracle with zero recurrent weights
for LIN_GRU; closed forms (constant gates, saturated gates, resets).
"""
import numpy as np

LIN_GRU, LIN_DECAY = 2, 3


def _f(x):
    if x is None:
        return None
    if hasattr(x, "detach"):
        x = x.detach().cpu().double().numpy()
    return np.asarray(x, dtype=np.float64)


def _sig(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0, e) / (1.0 + e)


def _sp(x):
    return np.maximum(x, 0) + np.log1p(np.exp(-np.abs(x)))


def lin_coef(cell, u, lam, bias, kappa=8.0):
    """(m, b) of h_t = (1 - m) h_{t-1} + b; u [..., G, D]."""
    p = _f(u) + (0 if bias is None else _f(bias))
    if cell == LIN_GRU:
        z = _sig(p[..., 0, :])
        return z, z * np.tanh(p[..., 1, :])
    w = kappa * _sp(_f(lam)) * _sig(p[..., 0, :])
    m = -np.expm1(-w)
    return m, np.sqrt(m * (2 - m)) * _sig(p[..., 1, :]) * p[..., 2, :]


def _keep(reset, shape):
    if reset is None:
        return np.ones(shape + (1,))
    r = reset.cpu().numpy() if hasattr(reset, "cpu") else np.asarray(reset)
    return 1.0 - (r != 0).astype(np.float64)[..., None]


def lin_seq(cell, u, lam=None, bias=None, h0=None, reset=None, kappa=8.0, delta=48 * 2.0 ** -24):
    """States h [B, T, D], and a bound on an fp32 evaluation's error: with m
    and b off by at most `delta` of themselves (for gate arguments up to 6:
    2.5 |x| + 9 roundings of a sigmoid, a dozen more for w, the series, the
    root and the products) and each state by three roundings of the terms that
    form it or its map, the error obeys
      E_t = (1 - m) E_{t-1} + delta (m |h_{t-1}| + |b|)
            + 6 2^-24 (|h_{t-1}| + |h_t| + |b|)."""
    m, b = lin_coef(cell, u, lam, bias, kappa)
    B, T, D = m.shape
    keep = _keep(reset, (B, T))
    h = np.zeros((B, D)) if h0 is None else _f(h0)
    e = np.zeros((B, D))
    H, E = np.empty((B, T, D)), np.empty((B, T, D))
    for t in range(T):
        h, e = h * keep[:, t], e * keep[:, t]
        n = (1 - m[:, t]) * h + b[:, t]
        e = ((1 - m[:, t]) * e + delta * (m[:, t] * np.abs(h) + np.abs(b[:, t]))
             + 6 * 2.0 ** -24 * (np.abs(h) + np.abs(n) + np.abs(b[:, t])))
        h = n
        H[:, t], E[:, t] = h, e
    return H, E


def lin_adjoint(cell, u, lam, bias, h0, h, g, reset=None, kappa=8.0, delta=48 * 2.0 ** -24):
    """{name: (gradient, error bound)} for du, dlam, dbias, dh0 along the
    given states h.  lambda's error obeys the states' recurrence in reverse;
    the factors of du are off by at most 2 delta of their magnitudes."""
    u, lam, bias, h, g = _f(u), _f(lam), _f(bias), _f(h), _f(g)
    B, T, D = h.shape
    keep = _keep(reset, (B, T))
    m, _ = lin_coef(cell, u, lam, bias, kappa)
    hp = np.concatenate([(np.zeros((B, D)) if h0 is None else _f(h0))[:, None], h[:, :-1]], 1) * keep
    L, E = np.empty_like(g), np.empty_like(g)
    mu, e = np.zeros((B, D)), np.zeros((B, D))
    for t in reversed(range(T)):
        L[:, t] = g[:, t] + mu
        E[:, t] = e + 2 * 2.0 ** -24 * (np.abs(g[:, t]) + np.abs(mu))
        mu = keep[:, t] * (1 - m[:, t]) * L[:, t]
        e = keep[:, t] * ((1 - m[:, t]) * E[:, t] + delta * m[:, t] * np.abs(L[:, t])
                          + 6 * 2.0 ** -24 * np.abs(L[:, t]))
    p = u + (0 if bias is None else bias)
    if cell == LIN_GRU:
        z, zc, c = _sig(p[..., 0, :]), _sig(-p[..., 0, :]), np.tanh(p[..., 1, :])
        t = np.exp(-2 * np.abs(p[..., 1, :]))       # 1 - tanh^2 of its own size: no cancellation is allowed for
        slope = z * 4 * t / (1 + t) ** 2
        f = np.stack([(c - hp) * z * zc, slope], 2)
        a = np.stack([(np.abs(c) + np.abs(hp)) * z * zc, slope], 2)
        ef = ea = None
    else:
        r, rc = _sig(p[..., 0, :]), _sig(-p[..., 0, :])
        i, ic, x = _sig(p[..., 1, :]), _sig(-p[..., 1, :]), p[..., 2, :]
        w = kappa * _sp(lam) * r
        beta, k = np.sqrt(m * (2 - m)), 1 - m
        ef = k * k * i * x * w / beta - k * hp * w
        ea = k * k * i * np.abs(x) * w / beta + k * np.abs(hp) * w
        f = np.stack([ef * rc, beta * x * i * ic, beta * i], 2)
        a = np.stack([ea * rc, np.abs(f[:, :, 1]), f[:, :, 2]], 2)
    du = L[:, :, None] * f
    edu = E[:, :, None] * np.abs(f) + 2 * delta * np.abs(L)[:, :, None] * a
    mag = np.abs(L)[:, :, None] * a
    depth = (T / 64 + B * 8 + 32) * 2.0 ** -24       # additions a value goes through, at most
    out = {"du": (du, edu), "dh0": (mu, e + 2.0 ** -24 * np.abs(mu)),
           "dbias": (du.sum((0, 1)), edu.sum((0, 1)) + depth * mag.sum((0, 1)))}
    if cell == LIN_DECAY:
        q = _sig(lam) / _sp(lam)
        out["dlam"] = (q * (L * ef).sum((0, 1)),
                       q * ((E * np.abs(ef) + (2 * delta + depth) * np.abs(L) * ea).sum((0, 1))))
    return out


# ------------------------------------------------------------ block norm --
def _act(kind, g):
    q, qc = _sig(g), _sig(-g)
    if kind == "silu":
        return g * q, q * (1 + g * qc), np.abs(g) * q, q * (1 + np.abs(g) * qc)
    return q, q * qc, q, q * qc


DELTA_NORM = 256 * 2.0 ** -24
"""Roundings of the block norm, forward or adjoint, as a share of the
magnitude: a mean of squares over threads that hold 8 or 16 channels (16 + 5 +
32 additions, half of it in the root), a gate of argument up to 8 (2.5 x 8 + 9
a time, at most three times), two such means and about 40 products and sums."""


def block_norm(h, gate=None, act="silu", w_post=None, res=None, scale=None, w_pre=None, eps=1e-6):
    """{name: (value, magnitude)} for s and x (x absent without w_pre)."""
    h, gate, w_post, res, scale, w_pre = map(_f, (h, gate, w_post, res, scale, w_pre))
    y, ya = h, np.abs(h)
    if w_post is not None:
        k = 1 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
        y, ya = y * k * w_post, ya * k * np.abs(w_post)
    if gate is not None:
        v, _, va, _ = _act(act, gate)
        y, ya = y * v, ya * va
    if scale is not None:
        y, ya = y * scale, ya * np.abs(scale)
    if res is not None:
        y, ya = y + res, ya + np.abs(res)
    out = {"s": (y, ya)}
    if w_pre is not None:
        k = 1 / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
        # an error e of s moves k by at most k^3 mean(|s| e)
        xa = k * np.abs(w_pre) * (ya + np.abs(y) * k * k * (np.abs(y) * ya).mean(-1, keepdims=True))
        out["x"] = (y * k * w_pre, xa)
    return out


def block_norm_adjoint(h, ds, dx, gate=None, act="silu", w_post=None, res=None, scale=None,
                       w_pre=None, eps=1e-6):
    """{name: (gradient, magnitude)} over rows h [N, D]; absent parts left out.
    The magnitudes of a norm's part count the root's change with its
    argument's error once more (the factor 2)."""
    h, ds, dx, gate, w_post, res, scale, w_pre = map(_f, (h, ds, dx, gate, w_post, res, scale, w_pre))
    one = np.ones(h.shape[-1])
    kh = 1 / np.sqrt((h * h).mean(-1, keepdims=True) + eps) if w_post is not None else 1.0
    hh, wp = h * kh, one if w_post is None else w_post
    v, dv, va, dva = (one, 0 * one, one, 0 * one) if gate is None else _act(act, gate)
    n = hh * wp
    y, ya = n * v, np.abs(n) * va
    sc = one if scale is None else scale
    r = 0 if res is None else res
    s, sa = r + sc * y, np.abs(r) + np.abs(sc) * ya
    out = {}
    d = np.zeros_like(h) if ds is None else ds
    da = np.abs(d)
    if w_pre is not None:
        k = 1 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
        cond = 1 + k * k * (np.abs(s) * sa).mean(-1, keepdims=True)
        sh, sha, e, ea = s * k, sa * k * cond, dx * w_pre, np.abs(dx * w_pre)
        out["dw_pre"] = ((dx * sh).sum(0), (np.abs(dx) * sha).sum(0))
        d = d + k * (e - sh * (e * sh).mean(-1, keepdims=True))
        da = da + k * cond * (ea + sha * (ea * sha).mean(-1, keepdims=True))
    if res is not None:
        out["dres"] = (d, da)
    if scale is not None:
        out["dscale"] = ((d * y).sum(0), (da * ya).sum(0))
    d, da = d * sc, da * np.abs(sc)
    if gate is not None:
        out["dgate"] = (d * n * dv, da * np.abs(n) * dva)
    d, da = d * v, da * va
    if w_post is not None:
        out["dw_post"] = ((d * hh).sum(0), (da * np.abs(hh)).sum(0))
        d, da = d * wp, da * np.abs(wp)
        d = kh * (d - hh * (d * hh).mean(-1, keepdims=True))
        da = 2 * kh * (da + np.abs(hh) * (da * np.abs(hh)).mean(-1, keepdims=True))
    out["dh"] = (d, da)
    return out
