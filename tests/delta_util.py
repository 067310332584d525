"""Inputs and bounds of the gated delta rule's and the layer norm's GPU tests."""
import math

import numpy as np

from gpu_util import torch_mod


def io_dtype(io):
    torch = torch_mod()
    return torch.bfloat16 if io == "bf16" else torch.float32


def delta_case(seed, b, l, h, g, n, p, io, normalize=False, packed=False, init=False, states=False,
               device="cuda", **over):
    """Inputs on the GPU (rounded to the io type) and what they were rounded to, in fp64."""
    torch = torch_mod()
    r = np.random.default_rng(seed)
    dt = io_dtype(io)

    def put(a, dtype=dt):
        return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(device).to(dtype)
    q, k = r.normal(size=(b, l, g, n)), r.normal(size=(b, l, g, n))
    if not normalize:
        k /= np.sqrt((k * k).sum(-1, keepdims=True)) * 1.01  # rounding may not push it over 1
        q /= np.sqrt(n)
    at = np.exp(r.uniform(math.log(1e-3), math.log(0.1), size=h))
    f32 = torch.float32
    c = dict(q=put(q), k=put(k), v=put(r.normal(size=(b, l, h, p))), dt=put(r.normal(size=(b, l, h))),
             A=put(-np.exp(r.uniform(0, math.log(16), size=h)), f32),
             beta=put(1 / (1 + np.exp(-r.normal(size=(b, l, h))))),
             dt_bias=put(np.log(np.expm1(at)), f32),
             init=put(r.normal(size=(b, h, n, p)) * 0.3, f32) if init else None, seq=None)
    if packed:
        c["seq"] = torch.from_numpy(np.cumsum(r.random((b, l)) < 0.04, 1).astype(np.int32)).to(device)
    c["dy"], c["d_final"] = put(r.normal(size=(b, l, h, p))), put(r.normal(size=(b, h, n, p)), f32)
    for name, f in over.items():
        c[name] = f(c[name])
    return c


def as64(c):
    return {k: None if v is None else (v.cpu().numpy() if k == "seq" else
                                       v.double().cpu().numpy()) for k, v in c.items()}


def rel(x, o):
    """Norm of the difference over the reference's norm; zero references are met exactly."""
    x = x.detach().double().cpu().numpy() if hasattr(x, "detach") else np.asarray(x, np.float64)
    assert x.shape == o.shape, (x.shape, o.shape)
    assert np.isfinite(x).all()
    o = np.where(np.abs(o) < 2.0 ** -149, 0.0, o)  # what fp32 has no value for
    n = np.linalg.norm(o)
    d = np.linalg.norm(x - o)
    return 0.0 if d == 0 else math.inf if n == 0 else d / n


# Bounds on rel().  A rounding to bf16 is off by at most 2^-8 of the value, to
# fp16 2^-11; a two-term operand by 2^-22.
#   fp32 values of the recurrence: about six two-term operands follow each other
#   (S, k, R, T, U, k), and a contraction may gather errors of eight times its
#   result: 48 * 2^-22 < 1.2e-5.
#   decays' gradients: differences of sums of up to 64 such terms: eight times that.
#   y in bf16: its own rounding and three fp16 operands: 2^-8 + 3 * 2^-11.
#   dq, dk in bf16: their rounding, two operands' and the masked products': 4 * 2^-8.
FINE = 1.2e-5
DECAY = 8 * FINE
ONE = 2.0 ** -8 * 1.02
BOUNDS = {
    "f32": dict(y=FINE, state=FINE, dq=2 * FINE, dk=2 * FINE, dv=FINE, dbeta=2 * FINE, ddt=DECAY,
                dA=DECAY, ddt_bias=DECAY, d_init=FINE),
    "bf16": dict(y=2.0 ** -8 + 3 * 2.0 ** -11, state=FINE, dq=2.0 ** -6, dk=2.0 ** -6, dv=ONE,
                 dbeta=ONE, ddt=ONE, dA=DECAY, ddt_bias=DECAY, d_init=FINE),
}
