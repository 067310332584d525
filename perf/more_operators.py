"""Measured cases of the gated delta rule and of the layer norm in front of a
mixer, each with its gradient, and of the delta rule's decode step.

Operators (public entry points of mamba_ssd_chunked_chunk_amd):

    delta_scan      per head, with a state S [key_dim, value_dim]:
                        P_t = exp(A d_t) S_{t-1},  d_t = softplus(dt_t + dt_bias)
                        u_t = beta_t (v_t - P_t^T k_t)
                        S_t = P_t + k_t u_t^T,     y_t = scale S_t^T q_t
                    (k and q optionally divided by their norms first)
    delta_scan_bwd  its gradients
    delta_step      one token of it, the state updated in place
    layer_norm      s = x + residual, y = (s - mean) rstd weight + bias
    layer_norm_bwd  dx, dweight and dbias, with the residual stream's gradient added

With `own` false, run() computes them from elementary torch operations in
fp32, rounded once at the end; with `own` true it makes the framework's calls.
exact() computes the definitions in fp64, token by token.
"""
import math

import torch

own = False

CHUNK = 64  # tokens between the delta rule's saved states
NORM_EPS = 1e-6
LN_EPS = 1e-5

DT = {"bf16": torch.bfloat16, "f32": torch.float32}

# the largest scan (one row of 65536 tokens of 64 heads, 128 x 64) and the
# largest norm (16384 rows of 2560) bound the drawn cases
MOST_DELTA = 65536 * 64 * 128 * 64
MOST_NORM = 16384 * 2560


def listed():
    return [
        # a long context of one sequence, its final state kept
        dict(name="delta_long", op="delta_scan", b=1, l=65536, h=64, g=8, n=128, p=64, io="bf16",
             norm=False, packed=False, init=False, final=True, states=False),
        # a training batch: keys normalised in the call, states kept for the gradient
        dict(name="delta_train", op="delta_scan", b=8, l=2048, h=24, g=24, n=128, p=64, io="bf16",
             norm=True, packed=False, init=False, final=False, states=True),
        # prompts of ragged length continued from states, two value heads to a key head
        dict(name="delta_prompt", op="delta_scan", b=16, l=1000, h=16, g=8, n=128, p=128, io="bf16",
             norm=True, packed=False, init=True, final=True, states=False),
        # packed documents, fp32, odd lengths
        dict(name="delta_packed_f32", op="delta_scan", b=2, l=509, h=6, g=3, n=64, p=32, io="f32",
             norm=False, packed=True, init=False, final=True, states=False),
        # the gradient over a training batch, from the states that the forward pass kept
        dict(name="delta_bwd_train", op="delta_scan_bwd", b=4, l=2048, h=16, g=16, n=128, p=128,
             io="bf16", norm=True, packed=False, init=False, final=False, states=True),
        # the gradient of packed documents in fp32, no states kept, from an initial state
        dict(name="delta_bwd_packed_f32", op="delta_scan_bwd", b=3, l=333, h=4, g=2, n=32, p=64,
             io="f32", norm=False, packed=True, init=True, final=True, states=False),
        # a decode step of 256 sequences
        dict(name="delta_step_256", op="delta_step", b=256, h=80, g=8, n=128, p=64, io="bf16",
             norm=True),
        # a decode step of one sequence: latency
        dict(name="delta_step_1", op="delta_step", b=1, h=24, g=24, n=128, p=64, io="f32",
             norm=False),
        # the norm in front of a mixer over a training batch, with the block's residual
        dict(name="norm_train", op="layer_norm", m=16384, n=2560, io="bf16", residual=True),
        # the same of one decoded token: latency
        dict(name="norm_token", op="layer_norm", m=1, n=2560, io="bf16", residual=True),
        # its gradient over a training batch
        dict(name="norm_bwd_train", op="layer_norm_bwd", m=16384, n=2560, io="bf16",
             residual=True),
        # the gradient in fp32 at odd sizes
        dict(name="norm_bwd_odd_f32", op="layer_norm_bwd", m=1999, n=771, io="f32",
             residual=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["delta_scan", "delta_scan", "delta_scan_bwd", "delta_scan_bwd", "delta_step",
                     "layer_norm", "layer_norm_bwd"])
    io = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("layer_norm", "layer_norm_bwd"):
        n = _log(rng, 16, 10576)
        if rng.random() < 0.6:  # most layers' widths are multiples of 16
            n = max(16, n // 16 * 16)
        m = max(1, min(_log(rng, 1, 65536), MOST_NORM // (2 if io == "f32" else 1) // n))
        return dict(op=op, m=m, n=n, io=io, residual=rng.random() < 0.5)
    g = rng.choice([1, 2, 3, 4, 8, 16])
    h = min(64, g * rng.choice([1, 1, 2, 3, 4]))
    n, p = rng.choice([32, 64, 128, 128]), rng.choice([16, 32, 64, 64, 128, 128])
    norm = rng.random() < 0.6
    if op == "delta_step":
        b = _log(rng, 1, 256)
        return dict(op=op, b=b, h=h, g=g, n=n, p=p, io=io, norm=norm)
    bwd = op == "delta_scan_bwd"
    b, l = _log(rng, 1, 16), _log(rng, 1, 4096 if bwd else 65536)
    most = MOST_DELTA // (8 if bwd else 1) // (4 if io == "f32" else 1)
    l = max(1, min(l, most // (b * h * n * p)))
    return dict(op=op, b=b, l=l, h=h, g=g, n=n, p=p, io=io, norm=norm, packed=rng.random() < 0.4,
                init=rng.random() < 0.5, final=rng.random() < 0.5, states=rng.random() < 0.5)


def work(case):
    e = 2 if case["io"] == "bf16" else 4
    op = case["op"]
    if op == "layer_norm":
        el, rows = case["m"] * case["n"], 4 if case["residual"] else 2
        return {"bytes": e * rows * el + 8 * case["n"] + 8 * case["m"], "flops": 8 * el}
    if op == "layer_norm_bwd":
        el, rows = case["m"] * case["n"], 4 if case["residual"] else 3
        return {"bytes": e * rows * el + 12 * case["n"] + 8 * case["m"], "flops": 14 * el}
    b, h, g, n, p = (case[k] for k in "bhgnp")
    state = 4 * b * h * n * p
    if op == "delta_step":
        return {"bytes": 2 * state + e * b * (2 * g * n + 2 * h * p + 2 * h) + 8 * h,
                "flops": 7 * b * h * n * p}
    l = case["l"]
    kept = state * -(-l // CHUNK) * int(case["states"])
    side = 4 * b * l * int(case["packed"]) + 8 * h + kept
    if op == "delta_scan":
        ends = state * (int(case["init"]) + int(case["final"]))
        return {"bytes": e * b * l * (2 * g * n + 2 * h * p + 2 * h) + side + ends,
                "flops": 7 * b * l * h * n * p}
    ends = state * (2 * int(case["init"]) + int(case["final"]))
    return {"bytes": e * b * l * (4 * g * n + 3 * h * p + 4 * h) + side + 8 * h + ends,
            "flops": 16 * b * l * h * n * p}


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

    io, op = DT[case["io"]], case["op"]
    s = dict(case)
    if op in ("layer_norm", "layer_norm_bwd"):
        m, n = case["m"], case["n"]
        s["w"], s["bias"] = 1 + normal(n, std=0.2), normal(n, std=0.2)
        s["x"] = normal(m, n, dtype=io)
        if op == "layer_norm":
            s["r"] = normal(m, n, std=2.0, dtype=io) if case["residual"] else None
            return s
        s["dy"] = normal(m, n, dtype=io)
        s["dsum"] = normal(m, n, dtype=io) if case["residual"] else None
        x = s["x"].float()  # what the forward pass left
        mean = x.mean(-1)
        var = ((x - mean[:, None]) ** 2).mean(-1)
        s["stats"] = torch.stack([mean, 1 / torch.sqrt(var + LN_EPS)])
        return s
    b, h, g, n, p = (case[k] for k in "bhgnp")
    lead = (b,) if op == "delta_step" else (b, case["l"])
    q, k = normal(*lead, g, n), normal(*lead, g, n)
    if not case["norm"]:  # normalised by the program, before the call
        q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + NORM_EPS)
        k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + NORM_EPS)
    s["q"], s["k"], s["v"] = q.to(io), k.to(io), normal(*lead, h, p, dtype=io)
    s["dt"], s["beta"] = normal(*lead, h, dtype=io), torch.sigmoid(normal(*lead, h)).to(io)
    s["A"] = -torch.exp(math.log(16.0) * torch.rand(h, generator=gen, device=dev))
    at = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(h, generator=gen, device=dev))
    s["dt_bias"] = torch.log(torch.expm1(at))
    s["scale"] = 1.0 / math.sqrt(n)
    if op == "delta_step":
        s["state"] = normal(b, h, n, p, std=0.3)
        return s
    s["h0"] = normal(b, h, n, p, std=0.3) if case["init"] else None
    s["seq"] = _documents(b, case["l"], gen, dev) if case["packed"] else None
    if op == "delta_scan_bwd":
        s["dy"] = normal(*lead, h, p, dtype=io)
        s["dfin"] = normal(b, h, n, p, std=0.1) if case["final"] else None
        s["kept"] = None
        if case["states"]:  # what the forward pass left: the state after every CHUNK tokens
            s["kept"] = _delta_states(s, _delta_terms(s))[1].transpose(0, 1)[:, 1:].contiguous()
    return s


# ------------------------------------------------------------ plain forms --
def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def _unit(s, t):
    """q or k in fp32, divided by its norm where the call does that, and 1 / norm."""
    t = t.float()
    if not s["norm"]:
        return t, None
    r = 1 / torch.sqrt((t * t).sum(-1, keepdim=True) + NORM_EPS)
    return t * r, r


def _chunks(t, l, heads=None):
    """[b, l, ...] -> [chunks, b, (heads,) CHUNK, ...], zeros behind the last token."""
    pad = -l % CHUNK
    if pad:
        t = torch.cat([t, torch.zeros_like(t[:, :1]).expand(-1, pad, *t.shape[2:])], 1)
    t = t.reshape(t.shape[0], -1, CHUNK, *t.shape[2:]).transpose(0, 1)
    if heads is None:
        return t
    t = t.transpose(2, 3)  # [chunks, b, heads, CHUNK, ..]
    return t.repeat_interleave(heads // t.shape[2], 2)


def _delta_terms(s):
    """Everything of the chunks that does not depend on the state."""
    l, h = s["l"], s["h"]
    q, rq = _unit(s, s["q"])
    k, rk = _unit(s, s["k"])
    z = s["dt"].float() + s["dt_bias"]
    d = _softplus(z)
    t = dict(rq=rq, rk=rk, z=z, d=d, q=_chunks(q, l, h), k=_chunks(k, l, h),
             v=_chunks(s["v"].float(), l, h), beta=_chunks(s["beta"].float(), l, h)[..., None])
    at = torch.cumsum(_chunks(d.double() * s["A"].double(), l, h), -1)  # log decays add up in fp64
    seq = s.get("seq")
    own_doc = torch.zeros((s["b"], l), dtype=torch.int64, device=z.device) if seq is None else seq
    new = torch.zeros_like(own_doc, dtype=torch.bool)
    new[:, 1:] = own_doc[:, 1:] != own_doc[:, :-1]
    count = torch.cumsum(new.long(), 1)
    count = torch.cat([count, count[:, -1:].expand(-1, -l % CHUNK)], 1)
    doc = count.reshape(s["b"], -1, CHUNK).transpose(0, 1)[:, :, None]       # [chunks, b, 1, CHUNK]
    before = torch.cat([torch.zeros_like(doc[:1, ..., -1]), doc[:-1, ..., -1]])[..., None]
    none = torch.zeros((), dtype=torch.float64, device=z.device)
    lower = torch.ones((CHUNK, CHUNK), dtype=torch.bool, device=z.device).tril()
    span = (at[..., :, None] - at[..., None, :]).masked_fill(~lower, -math.inf)
    decay = torch.where(doc[..., :, None] == doc[..., None, :], torch.exp(span), none).float()
    last, end = doc[..., -1:], at[..., -1:]
    t["read"] = torch.where(doc == before, torch.exp(at), none).float()[..., None]
    t["write"] = torch.where(doc == last, torch.exp(end - at), none).float()[..., None]
    t["carry"] = torch.where(last == before, torch.exp(end), none).float()[..., None]
    t["new"] = new
    kt = t["k"].transpose(-1, -2)
    t["decay"] = decay
    t["kk"] = (t["k"] @ kt) * decay * lower.tril(-1)
    t["qk"] = (t["q"] @ kt) * decay
    # rows of (I + kk diag(beta))^-1, one after the other
    m = -t["kk"] * t["beta"].transpose(-1, -2)
    for i in range(1, CHUNK):
        m[..., i, :i] += (m[..., i, :i, None] * m[..., :i, :i]).sum(-2)
    t["solve"] = m + torch.eye(CHUNK, device=m.device)
    return t


def _delta_states(s, t):
    """v - P^T k of every token, and the state in front of every chunk and after the last."""
    b, h, n, p = (s[x] for x in "bhnp")
    state = torch.zeros((b, h, n, p), device=t["k"].device) if s["h0"] is None else s["h0"]
    ns, states = [], [state]
    wk, rk = (t["k"] * t["write"]).transpose(-1, -2), t["k"] * t["read"]
    for c in range(t["k"].shape[0]):
        ns.append(t["solve"][c] @ (t["v"][c] - rk[c] @ state))
        state = t["carry"][c] * state + wk[c] @ (t["beta"][c] * ns[-1])
        states.append(state)
    return torch.stack(ns), torch.stack(states)


def _tokens(t, l):
    """[chunks, b, heads, CHUNK, ..] -> [b, l, heads, ..]."""
    t = t.transpose(0, 1).transpose(2, 3)
    return t.reshape(t.shape[0], -1, *t.shape[3:])[:, :l]


def _delta_scan(s):
    t, l = _delta_terms(s), s["l"]
    ns, states = _delta_states(s, t)
    y = s["scale"] * ((t["q"] * t["read"]) @ states[:-1] + t["qk"] @ (t["beta"] * ns))
    res = [_tokens(y, l).to(s["v"].dtype).contiguous()]
    if s["final"]:
        res.append(states[-1])
    if s["states"]:
        res.append(states[1:].transpose(0, 1).contiguous())
    return tuple(res)


def _unit_grad(g, t, r):
    return g if r is None else r * (g - (t.float() * r) * ((t.float() * r) * g).sum(-1, keepdim=True))


def _delta_bwd(s):
    t, l, h, g = _delta_terms(s), s["l"], s["h"], s["g"]
    ns, states = _delta_states(s, t)
    us = t["beta"] * ns
    dy = s["scale"] * _chunks(s["dy"].float(), l, h)
    nc = dy.shape[0]
    ds = torch.zeros_like(states[0]) if s["dfin"] is None else s["dfin"]
    after, drs, dus = [None] * nc, [None] * nc, [None] * nc
    into, wk = t["qk"].transpose(-1, -2) @ dy, t["k"] * t["write"]
    rq, rk = (t["q"] * t["read"]).transpose(-1, -2) @ dy, (t["k"] * t["read"]).transpose(-1, -2)
    back = t["solve"].transpose(-1, -2)
    for c in range(nc - 1, -1, -1):
        after[c] = ds
        dus[c] = into[c] + wk[c] @ ds
        drs[c] = back[c] @ (t["beta"][c] * dus[c])
        ds = t["carry"][c] * ds + rq[c] - rk[c] @ drs[c]
    after, dr, du = torch.stack(after), torch.stack(drs), torch.stack(dus)
    lower = torch.ones((CHUNK, CHUNK), dtype=torch.bool, device=ds.device).tril()
    dp = (dy @ us.transpose(-1, -2)) * lower
    da = -(dr @ us.transpose(-1, -2)) * lower.tril(-1)
    dbeta = ((du - t["kk"].transpose(-1, -2) @ dr) * ns).sum(-1)
    s0t = states[:-1].transpose(-1, -2)
    q_in, k_in = t["read"] * (dy @ s0t), -t["read"] * (dr @ s0t)
    k_out = t["write"] * (us @ after.transpose(-1, -2))
    both = da * t["decay"]
    dq = q_in + (dp * t["decay"]) @ t["k"]
    dk = k_in + k_out + (dp * t["decay"]).transpose(-1, -2) @ t["q"] \
        + (both + both.transpose(-1, -2)) @ t["k"]
    # the log decay up to token i: what it scales, less what it divides
    cell = (dp * t["qk"] + da * t["kk"]).double()
    out = (k_out * t["k"]).double().sum(-1)
    dat = (q_in * t["q"] + k_in * t["k"]).double().sum(-1) - out + cell.sum(-1) - cell.sum(-2)
    dat[..., -1] += out.sum(-1) + (t["carry"] * states[:-1] * after).double().sum((-1, -2))
    dlog = _tokens(torch.flip(torch.cumsum(torch.flip(dat, [-1]), -1), [-1]), l)
    new = t["new"]
    if s["h0"] is None:  # nothing in front of the first token either
        new = new.clone()
        new[:, 0] = True
    dlog = dlog.masked_fill(new[..., None], 0.0).float()
    dd = dlog * s["A"] * torch.sigmoid(t["z"])

    def groups(x, of, r):
        x = _tokens(x, l)
        x = x.reshape(*x.shape[:2], g, h // g, -1).sum(3)
        return _unit_grad(x, of, r).to(of.dtype)

    io = s["v"].dtype
    res = dict(dq=groups(dq, s["q"], t["rq"]), dk=groups(dk, s["k"], t["rk"]),
               dv=_tokens(dr, l).to(io).contiguous(), ddt=dd.to(io),
               dbeta=_tokens(dbeta, l).to(io).contiguous(), dA=(dlog * t["d"]).sum((0, 1)),
               ddt_bias=dd.sum((0, 1)))
    if s["h0"] is not None:
        res["d_init"] = ds
    return res


def _delta_step(s):
    ratio = s["h"] // s["g"]
    q = _unit(s, s["q"])[0].repeat_interleave(ratio, 1)
    k = _unit(s, s["k"])[0].repeat_interleave(ratio, 1)
    a = torch.exp(s["A"] * _softplus(s["dt"].float() + s["dt_bias"]))
    st = a[..., None, None] * s["state"]
    u = s["beta"].float()[..., None] * (s["v"].float() - (st * k[..., None]).sum(-2))
    s["state"].copy_(st + k[..., None] * u[:, :, None])
    return (s["scale"] * (s["state"] * q[..., None]).sum(-2)).to(s["v"].dtype), s["state"]


def _layer_norm(s):
    x = s["x"]
    if s["r"] is not None:
        x = (x.float() + s["r"].float()).to(x.dtype)
    f = x.float()
    mean = f.mean(-1)
    c = f - mean[:, None]
    rstd = 1 / torch.sqrt((c * c).mean(-1) + LN_EPS)
    y = (c * rstd[:, None] * s["w"] + s["bias"]).to(x.dtype)
    return ((y,) if s["r"] is None else (y, x)) + (torch.stack([mean, rstd]),)


def _layer_norm_bwd(s):
    mean, rstd = s["stats"][0][:, None], s["stats"][1][:, None]
    hat, dy = (s["x"].float() - mean) * rstd, s["dy"].float()
    g = dy * s["w"]
    dx = rstd * (g - g.mean(-1, keepdim=True) - hat * (g * hat).mean(-1, keepdim=True))
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return dict(dx=dx.to(s["x"].dtype), dweight=(dy * hat).sum(0), dbias=dy.sum(0))


def run(state):
    s = state
    op = s["op"]
    if not own:
        return {"delta_scan": _delta_scan, "delta_scan_bwd": _delta_bwd, "delta_step": _delta_step,
                "layer_norm": _layer_norm, "layer_norm_bwd": _layer_norm_bwd}[op](s)
    import mamba_ssd_chunked_chunk_amd as ssd
    if op == "layer_norm":
        return ssd.layer_norm(s["x"], s["w"], s["bias"], residual=s["r"], eps=LN_EPS,
                              return_stats=True)
    if op == "layer_norm_bwd":
        return ssd.layer_norm_bwd(s["dy"], s["x"], s["stats"], s["w"], bias=True,
                                  d_sum=s["dsum"])
    kw = dict(dt_bias=s["dt_bias"], scale=s["scale"], normalize=s["norm"], norm_eps=NORM_EPS)
    if op == "delta_step":
        return ssd.delta_step(s["state"], s["q"], s["k"], s["v"], s["dt"], s["A"], s["beta"],
                              **kw), s["state"]
    kw.update(initial_state=s["h0"], seq_idx=s["seq"])
    if op == "delta_scan":
        y = ssd.delta_scan(s["q"], s["k"], s["v"], s["dt"], s["A"], s["beta"],
                           return_final_state=s["final"], return_states=s["states"], **kw)
        return y if isinstance(y, tuple) else (y,)
    return ssd.delta_scan_bwd(s["q"], s["k"], s["v"], s["dt"], s["A"], s["beta"], s["dy"],
                              d_final=s["dfin"], states=s["kept"], **kw)


# ----------------------------------------------------------------- exact --
def _wide(t):
    return t.double()


def _exact_norm(case, s):
    x = _wide(s["x"])
    if case["op"] == "layer_norm":
        if s["r"] is not None:
            x = _wide((x + _wide(s["r"])).to(s["x"].dtype))
        mean, var = x.mean(1), x.var(1, unbiased=False)
        y = torch.addcmul(_wide(s["bias"]), (x - mean[:, None]) / torch.sqrt(var + LN_EPS)[:, None],
                          _wide(s["w"]))
        st = torch.stack([mean, torch.rsqrt(var + LN_EPS)])
        return (y, st) if s["r"] is None else (y, x, st)
    # row by row as the Jacobian (rstd / n) (n I - 1 1^T - hat hat^T) applied to w dy
    n, rstd = x.shape[1], _wide(s["stats"][1])
    hat = torch.addcmul(-(_wide(s["stats"][0]) * rstd)[:, None], x, rstd[:, None])
    dy = _wide(s["dy"])
    e = dy * _wide(s["w"])
    dx = (n * e - e.sum(1)[:, None] - hat * torch.einsum("mn,mn->m", e, hat)[:, None]) \
        * (rstd / n)[:, None]
    if s["dsum"] is not None:
        dx += _wide(s["dsum"])
    return dict(dx=dx, dweight=torch.einsum("mn,mn->n", dy, hat),
                dbias=torch.mv(dy.t(), torch.ones_like(rstd)))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("layer_norm", "layer_norm_bwd"):
        return _exact_norm(case, s)
    b, h, g, n, p = (case[k] for k in "bhgnp")
    A, bias, scale, dev = _wide(s["A"]), _wide(s["dt_bias"]), s["scale"], s["q"].device
    at = (lambda x, t: x) if op == "delta_step" else (lambda x, t: x[:, t])
    seq = s.get("seq")

    def unit(x):
        x = _wide(x)
        r = (x.square().sum(-1, keepdim=True) + NORM_EPS).rsqrt() if case["norm"] \
            else torch.ones_like(x[..., :1])
        return x * r, r

    def heads(x):
        return x[:, :, None].expand(b, g, h // g, n).reshape(b, h, n)

    def token(t):
        """Kept share, update's strength, key, query and value of token t, per head."""
        step = torch.logaddexp(_wide(at(s["dt"], t)) + bias, torch.zeros_like(bias))
        keep = torch.exp(A * step)
        if seq is not None and t > 0:
            keep = keep * (seq[:, t] == seq[:, t - 1])[:, None]
        return keep, _wide(at(s["beta"], t)), heads(unit(at(s["k"], t))[0]), \
            heads(unit(at(s["q"], t))[0]), _wide(at(s["v"], t))

    def forward(S, t):
        keep, beta, k, q, v = token(t)
        held = S * keep[..., None, None]
        miss = v - torch.matmul(k[:, :, None], held)[:, :, 0]
        u = beta[..., None] * miss
        return torch.addcmul(held, k[..., None], u[:, :, None]), held, miss, u, keep, beta, k, q

    if op == "delta_step":
        S = forward(_wide(s["state"]), 0)
        return scale * torch.matmul(S[7][:, :, None], S[0])[:, :, 0], S[0]
    l = case["l"]
    # each token takes about a dozen passes over the state in front, three dozen in the gradient
    if b * h * n * p * l * (3 if op == "delta_scan_bwd" else 1) > 5e10 \
            or (op == "delta_scan_bwd" and l > 20000):
        return None
    S = torch.zeros((b, h, n, p), dtype=torch.float64, device=dev) if s["h0"] is None \
        else _wide(s["h0"])
    if op == "delta_scan":
        y = torch.empty((b, l, h, p), dtype=torch.float64, device=dev)
        kept = []
        for t in range(l):
            f = forward(S, t)
            S = f[0]
            y[:, t] = scale * torch.matmul(f[7][:, :, None], S)[:, :, 0]
            if case["states"] and (t % CHUNK == CHUNK - 1 or t == l - 1):
                kept.append(S)
        return (y,) + ((S,) if case["final"] else ()) \
            + ((torch.stack(kept, 1),) if case["states"] else ())
    starts = []
    for t in range(l):
        if t % CHUNK == 0:
            starts.append(S)
        S = forward(S, t)[0]
    D = torch.zeros_like(S) if s["dfin"] is None else _wide(s["dfin"])
    new = lambda *sh: torch.zeros(sh, dtype=torch.float64, device=dev)  # noqa: E731
    dq, dk, dv, dlog, dbeta = new(b, l, g, n), new(b, l, g, n), new(b, l, h, p), new(b, l, h), \
        new(b, l, h)
    for c in range(len(starts) - 1, -1, -1):
        run_, S = [], starts[c]
        for t in range(c * CHUNK, min(l, (c + 1) * CHUNK)):
            run_.append(forward(S, t))
            S = run_[-1][0]
        for t in range(min(l, (c + 1) * CHUNK) - 1, c * CHUNK - 1, -1):
            S, held, miss, u, keep, beta, k, q = run_.pop()
            e = scale * _wide(s["dy"][:, t])
            dq[:, t] = torch.matmul(S, e[..., None])[..., 0].reshape(b, g, -1, n).sum(2)
            D = torch.addcmul(D, q[..., None], e[:, :, None])
            gu = torch.matmul(k[:, :, None], D)[:, :, 0]
            dbeta[:, t] = (gu * miss).sum(-1)
            gv = beta[..., None] * gu
            dv[:, t] = gv
            dk[:, t] = (torch.matmul(D, u[..., None]) - torch.matmul(held, gv[..., None]))[
                ..., 0].reshape(b, g, -1, n).sum(2)
            D = torch.addcmul(D, k[..., None], gv[:, :, None], value=-1)
            dlog[:, t] = (D * held).sum((-1, -2))
            D = D * keep[..., None, None]
    for grad, of in ((dq, s["q"]), (dk, s["k"])):
        if case["norm"]:
            hat, r = unit(of)
            grad.copy_(r * (grad - hat * (hat * grad).sum(-1, keepdim=True)))
    z = _wide(s["dt"]) + bias
    dstep = dlog * A * torch.special.expit(z)
    res = dict(dq=dq, dk=dk, dv=dv, ddt=dstep, dbeta=dbeta,
               dA=(dlog * torch.logaddexp(z, torch.zeros_like(z))).sum((0, 1)),
               ddt_bias=dstep.sum((0, 1)))
    if s["h0"] is not None:
        res["d_init"] = D
    return res
