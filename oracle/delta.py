"""fp64 oracle of the gated delta rule, its gradient and its step, token by
token, and of the layer norm with its gradient."""
from __future__ import annotations

import math

import numpy as np
from scipy.special import expit

CHUNK = 64


def _unit(x, normalize, eps):
    x = np.asarray(x, np.float64)
    if not normalize:
        return x, np.ones(x.shape[:-1] + (1,))
    ss = (x * x).sum(-1, keepdims=True)
    ss = ss + eps
    r = np.where(ss > 0, 1 / np.sqrt(np.where(ss > 0, ss, 1.0)), 0.0)
    return x * r, r


def _steps(dt, bias, softplus, limit):
    z = np.asarray(dt, np.float64) + (0.0 if bias is None else np.asarray(bias, np.float64))
    sp = np.logaddexp(z, 0.0) if softplus else z
    d = np.clip(sp, limit[0], limit[1])
    slope = ((sp >= limit[0]) & (sp <= limit[1])) * (expit(z) if softplus else 1.0)
    return d, slope


def _setup(q, k, v, dt, A, beta, dt_bias, dt_softplus, dt_limit, scale, normalize, norm_eps, seq):
    v, beta, A = (np.asarray(t, np.float64) for t in (v, beta, A))
    h, (g, n) = v.shape[-2], np.asarray(k).shape[-2:]
    kh, rk = _unit(k, normalize, norm_eps)
    qh, rq = _unit(q, normalize, norm_eps)
    d, slope = _steps(dt, dt_bias, dt_softplus, dt_limit)
    keep = np.exp(A * d)
    cut = np.zeros(keep.shape, bool)
    if seq is not None:
        cut[:, 1:] = (seq[:, 1:] != seq[:, :-1])[..., None]
    keep = np.where(cut, 0.0, keep)
    rep = lambda t: np.repeat(t, h // g, axis=-2)  # noqa: E731
    return dict(q=rep(qh), k=rep(kh), qh=qh, kh=kh, rq=rq, rk=rk, v=v, beta=beta, A=A, d=d,
                slope=slope, keep=keep, scale=n ** -0.5 if scale is None else scale, h=h, g=g, n=n,
                p=v.shape[-1])


def _token(s, S, t):
    P = s["keep"][:, t, :, None, None] * S
    miss = s["v"][:, t] - np.einsum("bhnp,bhn->bhp", P, s["k"][:, t])
    u = s["beta"][:, t, :, None] * miss
    return P, miss, u, P + s["k"][:, t, :, :, None] * u[:, :, None, :]


def scan(q, k, v, dt, A, beta, dt_bias=None, dt_softplus=True, dt_limit=(0.0, math.inf),
         scale=None, normalize=False, norm_eps=1e-6, init=None, seq=None):
    """dict y [b, l, h, p], final [b, h, n, p], states (after every CHUNK tokens)."""
    s = _setup(q, k, v, dt, A, beta, dt_bias, dt_softplus, dt_limit, scale, normalize, norm_eps, seq)
    b, l = s["v"].shape[:2]
    S = np.zeros((b, s["h"], s["n"], s["p"])) if init is None else np.asarray(init, np.float64)
    y, states = np.empty_like(s["v"]), []
    for t in range(l):
        S = _token(s, S, t)[3]
        y[:, t] = s["scale"] * np.einsum("bhnp,bhn->bhp", S, s["q"][:, t])
        if t % CHUNK == CHUNK - 1 or t == l - 1:
            states.append(S)
    return dict(y=y, final=S, states=np.stack(states, 1) if states else None)


def grad(q, k, v, dt, A, beta, dy, dt_bias=None, dt_softplus=True, dt_limit=(0.0, math.inf),
         scale=None, normalize=False, norm_eps=1e-6, init=None, seq=None, d_final=None):
    """Gradients of sum(dy y) + sum(d_final final), as the binding returns them."""
    s = _setup(q, k, v, dt, A, beta, dt_bias, dt_softplus, dt_limit, scale, normalize, norm_eps, seq)
    b, l = s["v"].shape[:2]
    S = np.zeros((b, s["h"], s["n"], s["p"])) if init is None else np.asarray(init, np.float64)
    kept = []
    for t in range(l):
        kept.append((S,) + _token(s, S, t))
        S = kept[-1][4]
    D = np.zeros_like(S) if d_final is None else np.asarray(d_final, np.float64).copy()
    dq, dk = np.zeros_like(s["q"]), np.zeros_like(s["k"])
    dv, dlog, dbeta = np.zeros_like(s["v"]), np.zeros(s["keep"].shape), np.zeros(s["keep"].shape)
    for t in range(l - 1, -1, -1):
        S0, P, miss, u, S1 = kept[t]
        e = s["scale"] * np.asarray(dy, np.float64)[:, t]
        dq[:, t] = np.einsum("bhnp,bhp->bhn", S1, e)
        D = D + s["q"][:, t, :, :, None] * e[:, :, None, :]
        gu = np.einsum("bhnp,bhn->bhp", D, s["k"][:, t])
        dbeta[:, t] = (gu * miss).sum(-1)
        gv = s["beta"][:, t, :, None] * gu
        dv[:, t] = gv
        dk[:, t] = np.einsum("bhnp,bhp->bhn", D, u) - np.einsum("bhnp,bhp->bhn", P, gv)
        D = D - s["k"][:, t, :, :, None] * gv[:, :, None, :]
        dlog[:, t] = (D * P).sum((-1, -2))
        D = s["keep"][:, t, :, None, None] * D
    group = lambda t: t.reshape(b, l, s["g"], -1, s["n"]).sum(3)  # noqa: E731

    def through(gr, hat, r):
        return r * (gr - hat * (hat * gr).sum(-1, keepdims=True)) if normalize else gr
    ddt = dlog * s["A"] * s["slope"]
    res = dict(dq=through(group(dq), s["qh"], s["rq"]), dk=through(group(dk), s["kh"], s["rk"]),
               dv=dv, ddt=ddt, dbeta=dbeta, dA=(dlog * s["d"]).sum((0, 1)))
    if dt_bias is not None:
        res["ddt_bias"] = ddt.sum((0, 1))
    if init is not None:
        res["d_init"] = D
    return res


def step(state, q, k, v, dt, A, beta, **kw):
    """(y, new state) of one token."""
    one = lambda t: np.asarray(t)[:, None]  # noqa: E731
    r = scan(one(q), one(k), one(v), one(dt), A, one(beta), init=state, **kw)
    return r["y"][:, 0], r["final"]


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """(y, mean, rstd) over the last axis."""
    x = np.asarray(x, np.float64)
    mean = x.mean(-1)
    rstd = 1 / np.sqrt(((x - mean[..., None]) ** 2).mean(-1) + eps)
    y = (x - mean[..., None]) * rstd[..., None]
    return y * (1.0 if weight is None else np.asarray(weight, np.float64)) \
        + (0.0 if bias is None else np.asarray(bias, np.float64)), mean, rstd


def layer_norm_grad(dy, x, weight=None, eps=1e-5, d_sum=None):
    """dict dx, dweight, dbias."""
    hat, _, rstd = layer_norm(x, eps=eps)
    dy = np.asarray(dy, np.float64)
    g = dy * (1.0 if weight is None else np.asarray(weight, np.float64))
    dx = rstd[..., None] * (g - g.mean(-1, keepdims=True) - hat * (g * hat).mean(-1, keepdims=True))
    rows = tuple(range(dy.ndim - 1))
    return dict(dx=dx + (0.0 if d_sum is None else np.asarray(d_sum, np.float64)),
                dweight=(dy * hat).sum(rows), dbias=dy.sum(rows))
