"""fp64 oracle of the gated linear recurrence and its gradient, token by token,
with a first-order bound on what fp32 arithmetic may lose on the way."""
from __future__ import annotations

import numpy as np
from scipy.special import expit

CHUNK = 64


def _parts(x, gates, lam, scale, seq):
    x, gates = np.asarray(x, np.float64), np.asarray(gates, np.float64)
    lam = np.asarray(lam, np.float64)
    d = x.shape[-1]
    sp = np.logaddexp(lam, 0.0)
    sr, si = expit(gates[..., :d]), expit(gates[..., d:])
    u = scale * sp * sr
    a = np.exp(-u)
    beta = np.sqrt(-np.expm1(-2 * u))
    kept = a.copy()
    if seq is not None:
        kept[:, 1:][seq[:, 1:] != seq[:, :-1]] = 0.0
    return x, lam, sp, sr, si, u, a, beta, kept


def scan(x, gates, lam, scale, init=None, seq=None, delta=0.0):
    """dict y (= every state) [b, l, d], final [b, d], states; with `delta`, a
    relative error of every added value and (times max(1, u), as a relative
    error of u is u times as large in e^-u) of every decay, also err [b, l, d]:
    the error they bring to y."""
    x, lam, sp, sr, si, u, a, beta, kept = _parts(x, gates, lam, scale, seq)
    b, l, d = x.shape
    v = beta * si * x
    h = np.zeros((b, d)) if init is None else np.asarray(init, np.float64).copy()
    first = h.copy()
    big, e = np.abs(h), np.zeros((b, d))
    y, err = np.empty((b, l, d)), np.empty((b, l, d))
    du = delta * np.maximum(1.0, u)
    for t in range(l):
        e = kept[:, t] * e + du[:, t] * kept[:, t] * big + delta * np.abs(v[:, t])
        big = kept[:, t] * big + np.abs(v[:, t])
        h = kept[:, t] * h + v[:, t]
        y[:, t], err[:, t] = h, e
    at = [min(CHUNK * (c + 1), l) - 1 for c in range(-(-l // CHUNK))]
    return dict(y=y, final=h, states=y[:, at], err=err, first=first)


def grad(x, gates, lam, scale, dy, init=None, seq=None, d_final=None, delta=0.0):
    """dict dx, dgates, dlam, d_init, and with `delta` the error of each as
    err_dx, ... (first order in delta)."""
    fw = scan(x, gates, lam, scale, init, seq, delta)
    x, lam, sp, sr, si, u, a, beta, kept = _parts(x, gates, lam, scale, seq)
    b, l, d = x.shape
    dy = np.asarray(dy, np.float64)
    before = np.concatenate([fw["first"][:, None], fw["y"][:, :-1]], 1)
    ebefore = np.concatenate([np.zeros((b, 1, d)), fw["err"][:, :-1]], 1)
    q = np.zeros((b, d)) if d_final is None else np.asarray(d_final, np.float64).copy()
    big, e = np.abs(q), np.zeros((b, d))
    g, G, E = np.empty((b, l, d)), np.empty((b, l, d)), np.empty((b, l, d))
    du = delta * np.maximum(1.0, u)
    for t in range(l - 1, -1, -1):
        g[:, t] = dy[:, t] + q
        G[:, t] = np.abs(dy[:, t]) + big
        E[:, t] = e + delta * G[:, t]
        q = kept[:, t] * g[:, t]
        big = kept[:, t] * G[:, t]
        e = kept[:, t] * E[:, t] + du[:, t] * big
    ratio = np.where(u > 0, u / np.where(beta > 0, beta, 1.0), 0.0)
    w1, w2 = a * a * ratio * si * x, u * kept * before
    p = g * (w1 - w2)
    ep = E * (np.abs(w1) + np.abs(w2)) + np.abs(g) * u * kept * ebefore \
        + 4 * du * np.abs(g) * (np.abs(w1) + np.abs(w2))
    gi = g * beta * x * si * (1 - si)
    sig = np.where(lam < -30, 1.0, expit(lam) / sp)
    return dict(
        dx=g * beta * si, dgates=np.concatenate([p * (1 - sr), gi], -1),
        dlam=p.sum((0, 1)) * sig, d_init=q,
        err_dx=(E + 4 * delta * np.abs(g)) * beta * si,
        # one minus a sigmoid near one keeps an absolute error of delta
        err_dgates=np.concatenate(
            [ep * (1 - sr) + delta * np.abs(p),
             (E + 4 * delta * np.abs(g)) * beta * np.abs(x) * si * (1 - si)
             + delta * np.abs(g * beta * x * si)], -1),
        err_dlam=(ep + 4 * delta * np.abs(p)).sum((0, 1)) * sig,
        err_d_init=e)
