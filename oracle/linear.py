"""fp64 oracle of the products around a mixer: out = act(x W^T + b) + r and
its gradient."""
from __future__ import annotations

import math

import numpy as np
from scipy.special import expit, ndtr


def act(v, name):
    return {"none": lambda: v, "silu": lambda: v * expit(v), "gelu": lambda: v * ndtr(v),
            "sigmoid": lambda: expit(v)}[name]()


def act_grad(v, name):
    s = expit(v)
    return {"none": lambda: np.ones_like(v), "silu": lambda: s + v * s * expit(-v),
            "gelu": lambda: ndtr(v) + v * np.exp(-0.5 * v * v) / math.sqrt(2 * math.pi),
            "sigmoid": lambda: s * expit(-v)}[name]()


def linear(x, w, bias=None, activation="none", residual=None):
    """(out, pre) in fp64; x [m, k], w [n, k]."""
    pre = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T
    if bias is not None:
        pre = pre + np.asarray(bias, np.float64)
    out = act(pre, activation)
    if residual is not None:
        out = out + np.asarray(residual, np.float64)
    return out, pre


def linear_grad(dy, x, w, pre=None, activation="none"):
    """dict dx, dweight, dbias and e, the gradient at the pre-activation."""
    e = np.asarray(dy, np.float64)
    if activation != "none":
        e = e * act_grad(np.asarray(pre, np.float64), activation)
    return dict(e=e, dx=e @ np.asarray(w, np.float64), dweight=e.T @ np.asarray(x, np.float64),
                dbias=e.sum(0))
