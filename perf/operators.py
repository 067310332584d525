"""Measured cases of the products around a recurrent mixer and of its gated
linear recurrence.

Operators (public entry points of mamba_ssd_chunked_chunk_amd):

    linear          out = act(x W^T + bias) + residual           [.., K] -> [.., N]
    linear_bwd      dx, dW and dbias from dy and the saved pre-activation
    gated_scan      h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t per channel,
                    a_t = exp(-scale softplus(lam) sigmoid(r_t))
    gated_scan_bwd  its gradients
    gated_step      one token of it, the state updated in place

With `own` false, run() computes them from elementary torch operations in
fp32, rounded once at the end; with `own` true it makes the framework's calls.
exact() computes the definitions in fp64, token by token.
"""
import math

import torch

own = False

SCALE = 8.0
CHUNK = 64  # tokens between the recurrence's saved states

DT = {"bf16": torch.bfloat16, "f32": torch.float32}

# the largest product (16384 tokens through the 2.7b mixer's output projection)
# and the largest recurrence (one row of 65536 tokens) bound the drawn cases
MOST_MNK = 16384 * 5120 * 2560
MOST_SCAN = 65536 * 2560


def listed():
    return [
        # the output projection of a 2.7b mixer with the block's residual, over a training batch
        dict(name="linear_out_2p7b", op="linear", m=16384, k=5120, n=2560, io="bf16", act="none",
             bias=False, residual=True, pre=False),
        # the input projection of one decoded token of one sequence: bound by the weights' bytes
        dict(name="linear_token", op="linear", m=1, k=2560, n=10576, io="bf16", act="none",
             bias=False, residual=False, pre=False),
        # the output projection of a decode step of 256 sequences
        dict(name="linear_batch256", op="linear", m=256, k=5120, n=2560, io="bf16", act="none",
             bias=False, residual=True, pre=False),
        # an fp32 layer of a 130m block in training: bias, GELU, the pre-activation kept, ragged rows
        dict(name="linear_gelu_f32", op="linear", m=1999, k=768, n=1536, io="f32", act="gelu",
             bias=True, residual=True, pre=True),
        # the gradient of a 2.7b layer with GELU
        dict(name="linear_bwd_gelu", op="linear_bwd", m=8192, k=2560, n=5120, io="bf16",
             act="gelu", bias=True, residual=False, pre=False),
        # a gradient whose rows end off every vector width
        dict(name="linear_bwd_odd", op="linear_bwd", m=2047, k=770, n=1539, io="bf16",
             act="silu", bias=True, residual=False, pre=False),
        # a long context of one sequence, continued from a state
        dict(name="gated_scan_long", op="gated_scan", b=1, l=65536, d=2560, io="bf16", packed=False,
             init=True, states=False),
        # packed documents, fp32, odd sizes
        dict(name="gated_scan_packed_f32", op="gated_scan", b=2, l=509, d=771, io="f32", packed=True,
             init=False, states=True),
        # the gradient over a training batch, from the states that the forward pass kept
        dict(name="gated_scan_bwd_batch", op="gated_scan_bwd", b=4, l=4096, d=2560, io="bf16",
             packed=False, init=True, states=True),
        # the gradient of packed documents, no states kept
        dict(name="gated_scan_bwd_odd_f32", op="gated_scan_bwd", b=3, l=1001, d=771, io="f32",
             packed=True, init=False, states=False),
        # a decode step of 256 sequences
        dict(name="gated_step_256", op="gated_step", b=256, d=5120, io="bf16"),
        # a decode step of one sequence: latency
        dict(name="gated_step_1", op="gated_step", b=1, d=2560, io="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_bwd", "gated_scan", "gated_scan_bwd",
                     "gated_step"])
    io = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("linear", "linear_bwd"):
        bwd = op == "linear_bwd"
        m, k, n = _log(rng, 1, 16384), _log(rng, 32, 5120), _log(rng, 16, 10576)
        if rng.random() < 0.6:  # most layers' widths are multiples of 16
            k, n = max(16, k // 16 * 16), max(16, n // 16 * 16)
        most = MOST_MNK // (2 if bwd else 1) // (8 if io == "f32" else 1)
        m = max(1, min(m, most // (k * n)))
        act = rng.choice(["none", "none", "silu", "gelu", "sigmoid"])
        return dict(op=op, m=m, k=k, n=n, io=io, act=act, bias=rng.random() < 0.5,
                    residual=not bwd and rng.random() < 0.5,
                    pre=not bwd and act != "none" and rng.random() < 0.5)
    d = _log(rng, 32, 5120)
    if rng.random() < 0.6:
        d = max(16, d // 16 * 16)
    if op == "gated_step":
        return dict(op=op, b=_log(rng, 1, 512), d=d, io=io)
    b, l = _log(rng, 1, 16), _log(rng, 1, 65536)
    most = MOST_SCAN // (4 if op == "gated_scan_bwd" else 1)
    l = max(1, min(l, most // (b * d)))
    return dict(op=op, b=b, l=l, d=d, io=io, packed=rng.random() < 0.4, init=rng.random() < 0.5,
                states=rng.random() < 0.5)


def work(case):
    e = 2 if case["io"] == "bf16" else 4
    op = case["op"]
    if op in ("linear", "linear_bwd"):
        m, k, n = case["m"], case["k"], case["n"]
        if op == "linear":
            rows = 1 + int(case["residual"]) + int(case["pre"])
            return {"bytes": e * (m * k + n * k + rows * m * n) + 4 * n * int(case["bias"]),
                    "flops": 2 * m * n * k}
        rows = 2 if case["act"] != "none" else 1
        return {"bytes": e * (2 * m * k + 2 * n * k + rows * m * n) + 4 * n * int(case["bias"]),
                "flops": 4 * m * n * k}
    b, d = case["b"], case["d"]
    if op == "gated_step":
        return {"bytes": b * d * (4 * e + 8) + 4 * d, "flops": 20 * b * d}
    l = case["l"]
    el = b * l * d
    side = 4 * b * l * int(case["packed"]) + 4 * d + 4 * b * d * (1 + int(case["init"]))
    side += 4 * b * -(-l // CHUNK) * d * int(case["states"])
    if op == "gated_scan":
        return {"bytes": 4 * e * el + side, "flops": 20 * el}
    return {"bytes": 7 * e * el + side + 4 * d + 4 * b * d * int(case["init"]), "flops": 50 * el}


# ---------------------------------------------------------------- inputs --
def _documents(b, l, gen, dev):
    """Document index of every token: lengths around 100 tokens, single tokens among them."""
    cut = torch.rand((b, l), generator=gen, device=dev) < 0.01
    return torch.cumsum(cut.to(torch.int32), 1).to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(1_000_003 * (int(seed) + 1))

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=gen, device=dev) * std).to(dtype)

    io = DT[case["io"]]
    s = dict(case)
    if case["op"] in ("linear", "linear_bwd"):
        m, k, n = case["m"], case["k"], case["n"]
        s["x"] = normal(m, k, dtype=io)
        s["w"] = normal(n, k, std=1.0 / math.sqrt(k), dtype=io)
        if case["op"] == "linear":
            s["b"] = normal(n, std=0.5) if case["bias"] else None
            s["r"] = normal(m, n, dtype=io) if case["residual"] else None
        else:
            s["dy"] = normal(m, n, dtype=io)
            s["pre_in"] = normal(m, n, dtype=io) if case["act"] != "none" else None
        return s
    b, d = case["b"], case["d"]
    # decays exp(-scale softplus(lam)) spread over 0.9 .. 0.999, at a gate of one
    a = 0.9 + 0.099 * torch.rand(d, generator=gen, device=dev)
    s["lam"] = torch.log(torch.expm1(-torch.log(a) / SCALE)).to(torch.float32)
    if case["op"] == "gated_step":
        s["x"], s["gates"] = normal(b, d, dtype=io), normal(b, 2 * d, dtype=io)
        s["h"] = normal(b, d)
        return s
    l = case["l"]
    s["x"], s["gates"] = normal(b, l, d, dtype=io), normal(b, l, 2 * d, dtype=io)
    s["h0"] = normal(b, d) if case["init"] else None
    s["seq"] = _documents(b, l, gen, dev) if case["packed"] else None
    if case["op"] == "gated_scan_bwd":
        s["dy"], s["dfin"] = normal(b, l, d, dtype=io), normal(b, d)
        s["kept"] = None
        if case["states"]:  # what the forward pass left: the state after every CHUNK tokens
            h = _scan(*_terms(s)[:2], s["h0"])
            s["kept"] = _every(h, l)
            del h
    return s


def _every(h, l):
    at = torch.arange(CHUNK - 1, l + CHUNK - 1, CHUNK, device=h.device).clamp(max=l - 1)
    return h[:, at].contiguous()


# ------------------------------------------------------------ plain forms --
def _act(v, act):
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "sigmoid":
        return 1 / (1 + torch.exp(-v))
    return v


def _act_grad(v, act):
    if act == "silu":
        g = 1 / (1 + torch.exp(-v))
        return g * (1 + v * (1 - g))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(v * math.sqrt(0.5))) \
            + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)
    if act == "sigmoid":
        g = 1 / (1 + torch.exp(-v))
        return g * (1 - g)
    return torch.ones_like(v)


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def _terms(s):
    """Decay into each token (zero across documents), what it adds, and what the gradient needs."""
    d = s["lam"].shape[0]
    g = s["gates"].float()
    r, i = torch.sigmoid(g[..., :d]), torch.sigmoid(g[..., d:])
    u = SCALE * _softplus(s["lam"]) * r
    a = torch.exp(-u)
    beta = torch.sqrt(-torch.expm1(-2 * u))
    seq = s.get("seq")
    keep = a
    if seq is not None:
        same = torch.ones_like(seq, dtype=torch.bool)
        same[:, 1:] = seq[:, 1:] == seq[:, :-1]
        keep = torch.where(same[..., None], a, torch.zeros((), device=a.device))
    return keep, beta * i * s["x"].float(), r, i, u, a, beta


def _scan(a, v, h0):
    """h_t = a_t h_{t-1} + v_t along axis 1, by doubling the span that each entry covers."""
    a, v = a.clone(), v.clone()
    if h0 is not None:
        v[:, 0] += a[:, 0] * h0
    k = 1
    while k < v.shape[1]:
        v[:, k:] = v[:, k:] + a[:, k:] * v[:, :-k]
        a[:, k:] = a[:, k:] * a[:, :-k]
        k *= 2
    return v


def _plain(s):
    op, act = s["op"], s.get("act")
    if op == "linear":
        pre = s["x"].float() @ s["w"].float().t()
        if s["b"] is not None:
            pre = pre + s["b"]
        out = _act(pre, act)
        if s["r"] is not None:
            out = out + s["r"].float()
        out = out.to(s["x"].dtype)
        return (out, pre.to(s["x"].dtype)) if s["pre"] else out
    if op == "linear_bwd":
        g = s["dy"].float()
        if act != "none":
            g = g * _act_grad(s["pre_in"].float(), act)
        res = dict(dx=(g @ s["w"].float()).to(s["x"].dtype),
                   dweight=(g.t() @ s["x"].float()).to(s["x"].dtype))
        if s["bias"]:
            res["dbias"] = g.sum(0)
        return res
    a, v, r, i, u, a_own, beta = _terms(s)
    if op == "gated_step":
        s["h"].copy_(a * s["h"] + v)
        return s["h"].to(s["x"].dtype), s["h"]
    if op == "gated_scan":
        h = _scan(a, v, s["h0"])
        res = (h.to(s["x"].dtype), h[:, -1].contiguous())
        return res + ((_every(h, s["l"]),) if s["states"] else ())
    # the adjoint of the recurrence runs backwards: g_t = dy_t + a_{t+1} g_{t+1}
    h = _scan(a, v, s["h0"])
    before = torch.cat([(torch.zeros_like(h[:, :1]) if s["h0"] is None else s["h0"][:, None]),
                        h[:, :-1]], 1)
    dy = s["dy"].float()
    dy = torch.cat([dy[:, :-1], dy[:, -1:] + s["dfin"][:, None]], 1)
    nxt = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    g = _scan(nxt.flip(1), dy.flip(1), None).flip(1)
    x = s["x"].float()
    # u enters through the decay and through beta; u / beta stays finite as u goes to zero
    ratio = torch.where(u > 0, u / beta.clamp(min=1e-30), torch.zeros_like(u))
    by_log_u = g * (a_own * a_own * ratio * i * x - u * a * before)
    sp = _softplus(s["lam"])
    res = dict(dx=(g * beta * i).to(s["x"].dtype),
               dgates=torch.cat([by_log_u * (1 - r), g * beta * x * i * (1 - i)],
                                -1).to(s["x"].dtype),
               dlam=by_log_u.sum((0, 1)) * torch.sigmoid(s["lam"]) / sp)
    if s["h0"] is not None:
        res["d_init"] = a[:, 0] * g[:, 0]
    return res


def run(state):
    s = state
    if not own:
        return _plain(s)
    import mamba_ssd_chunked_chunk_amd as ssd
    op = s["op"]
    if op == "linear":
        return ssd.linear(s["x"], s["w"], bias=s["b"], activation=s["act"], residual=s["r"],
                          return_pre=s["pre"])
    if op == "linear_bwd":
        return ssd.linear_bwd(s["dy"], s["x"], s["w"], pre=s["pre_in"], activation=s["act"],
                              bias=s["bias"])
    if op == "gated_step":
        return ssd.gated_step(s["h"], s["x"], s["gates"], s["lam"], scale=SCALE), s["h"]
    if op == "gated_scan":
        return ssd.gated_scan(s["x"], s["gates"], s["lam"], scale=SCALE, initial_state=s["h0"],
                              seq_idx=s["seq"], return_final_state=True,
                              return_states=s["states"])
    return ssd.gated_scan_bwd(s["x"], s["gates"], s["lam"], s["dy"], scale=SCALE,
                              initial_state=s["h0"], d_final=s["dfin"], seq_idx=s["seq"],
                              states=s["kept"])


# ----------------------------------------------------------------- exact --
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]

    def wide(t):
        return t.double()

    if op in ("linear", "linear_bwd"):
        x, w, act = wide(s["x"]), wide(s["w"]), case["act"]
        half = math.sqrt(0.5)
        if op == "linear":
            z = torch.mm(x, w.t().contiguous())
            if s["b"] is not None:
                z += wide(s["b"])
            y = {"none": lambda: z.clone(), "silu": lambda: z * torch.special.expit(z),
                 "gelu": lambda: z * torch.special.ndtr(z),
                 "sigmoid": lambda: torch.special.expit(z)}[act]()
            if s["r"] is not None:
                y += wide(s["r"])
            return (y, z) if case["pre"] else y
        e = wide(s["dy"])
        if act != "none":
            z = wide(s["pre_in"])
            p = torch.special.expit(z)
            e = e * {"silu": lambda: p + z * p * torch.special.expit(-z),
                     "gelu": lambda: torch.special.ndtr(z)
                     + z * torch.exp(-(z * half) ** 2) / math.sqrt(2 * math.pi),
                     "sigmoid": lambda: p * torch.special.expit(-z)}[act]()
        res = dict(dx=torch.mm(e, w), dweight=torch.mm(e.t().contiguous(), x))
        if case["bias"]:
            res["dbias"] = torch.mv(e.t(), torch.ones(e.shape[0], dtype=e.dtype, device=e.device))
        return res

    d = case["d"]
    lam = wide(s["lam"])
    rate = SCALE * torch.logaddexp(lam, torch.zeros_like(lam))
    if op == "gated_step":
        g = wide(s["gates"])
        u = rate * torch.special.expit(g[:, :d])
        h = torch.exp(-u) * wide(s["h"]) \
            + torch.sqrt(-torch.special.expm1(-2 * u)) * torch.special.expit(g[:, d:]) * wide(s["x"])
        return h, h
    b, l = case["b"], case["l"]
    x, gates, seq = s["x"], s["gates"], s["seq"]
    new = None if seq is None else torch.cat(
        [torch.zeros_like(seq[:, :1]), (seq[:, 1:] != seq[:, :-1]).to(seq.dtype)], 1)

    def token(t):
        """Rate u, kept share and gates of token t, [b, d] each."""
        r = torch.special.expit(wide(gates[:, t, :d]))
        i = torch.special.expit(wide(gates[:, t, d:]))
        u = rate * r
        a = torch.exp(-u)
        kept = a if new is None else a * (1 - new[:, t, None])
        return r, i, u, a, kept, torch.sqrt(-torch.special.expm1(-2 * u))

    if l > 20000 and op == "gated_scan_bwd":
        return None
    h = wide(s["h0"]) if s["h0"] is not None else torch.zeros((b, d), dtype=torch.float64,
                                                              device=x.device)
    hs = torch.empty((b, l + 1, d), dtype=torch.float64, device=x.device)
    hs[:, 0] = h
    for t in range(l):
        r, i, u, a, kept, beta = token(t)
        h = kept * h + beta * i * wide(x[:, t])
        hs[:, t + 1] = h
    if op == "gated_scan":
        y = hs[:, 1:]
        res = (y, h)
        return res + ((torch.cat([y[:, CHUNK - 1::CHUNK], y[:, -1:]], 1)[:, :-(-l // CHUNK)],)
                      if case["states"] else ())
    dy, adj = s["dy"], wide(s["dfin"])
    dx = torch.empty((b, l, d), dtype=torch.float64, device=x.device)
    dg = torch.empty((b, l, 2 * d), dtype=torch.float64, device=x.device)
    drate = torch.zeros(d, dtype=torch.float64, device=x.device)
    for t in range(l - 1, -1, -1):
        r, i, u, a, kept, beta = token(t)
        adj = adj + wide(dy[:, t])
        xt = wide(x[:, t])
        du = adj * (i * xt * a * a / beta - kept * hs[:, t])
        dx[:, t] = adj * beta * i
        dg[:, t, :d] = du * u * (1 - r)
        dg[:, t, d:] = adj * beta * xt * i * (1 - i)
        drate += (du * r).sum(0)
        adj = kept * adj
    res = dict(dx=dx, dgates=dg, dlam=SCALE * drate * torch.special.expit(lam))
    if s["h0"] is not None:
        res["d_init"] = adj
    return res
