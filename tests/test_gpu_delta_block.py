"""The delta rule as a layer uses it: layer norm with the residual stream, one
projection to q, k, v and the gates, the delta rule, the gated norm and the
output projection -- forward, backward, one token at a time, and from a graph."""
import math

import numpy as np
import pytest

from gpu_util import log, torch_mod

pytestmark = pytest.mark.gpu

H, G, N, P = 4, 2, 32, 16
WIDTH = 2 * G * N + H * P


def _block(seed, dm, io):
    torch = torch_mod()
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    r = np.random.default_rng(seed)

    def t(*shape, std=1.0, dtype=dt):
        return torch.from_numpy((r.normal(size=shape) * std).astype(np.float32)).to("cuda").to(dtype)
    f = torch.float32
    return dict(nw=1 + t(dm, std=0.1, dtype=f), nb=t(dm, std=0.1, dtype=f),
                win=t(WIDTH, dm, std=dm ** -0.5), wdt=t(H, dm, std=dm ** -0.5),
                wb=t(H, dm, std=dm ** -0.5), bb=t(H, std=0.5, dtype=f),
                A=-torch.exp(t(H, dtype=f).abs()), dt_bias=t(H, dtype=f) - 3,
                wout=t(dm, H * P, std=(H * P) ** -0.5)), t


def _split(u):
    q, k, v = u.split([G * N, G * N, H * P], -1)
    lead = u.shape[:-1]
    return (q.reshape(*lead, G, N).contiguous(), k.reshape(*lead, G, N).contiguous(),
            v.reshape(*lead, H, P).contiguous())


def _front(ssd, p, x, res):
    y, s, st = ssd.layer_norm(x, p["nw"], p["nb"], residual=res, return_stats=True)
    beta, pre = ssd.linear(y, p["wb"], bias=p["bb"], activation="sigmoid", return_pre=True)
    return y, s, st, _split(ssd.linear(y, p["win"])), ssd.linear(y, p["wdt"]), beta, pre


def _forward(ssd, p, x, res, init):
    y, s, st, (q, k, v), dt, beta, pre = _front(ssd, p, x, res)
    o, fin, states = ssd.delta_scan(q, k, v, dt, p["A"], beta, dt_bias=p["dt_bias"], normalize=True,
                                    initial_state=init, return_final_state=True, return_states=True)
    out = ssd.linear(o.reshape(*o.shape[:2], H * P), p["wout"], residual=s)
    return out, fin, (y, s, st, q, k, v, dt, beta, pre, o, states)


def _backward(ssd, p, saved, init, dout):
    torch = torch_mod()
    y, s, st, q, k, v, dt, beta, pre, o, states = saved
    go = ssd.linear_bwd(dout, o.reshape(*o.shape[:2], H * P), p["wout"])
    g = ssd.delta_scan_bwd(q, k, v, dt, p["A"], beta, go["dx"].reshape(o.shape),
                           dt_bias=p["dt_bias"], normalize=True, initial_state=init, states=states)
    du = torch.cat([g[n].flatten(2) for n in ("dq", "dk", "dv")], -1)
    gi = ssd.linear_bwd(du, y, p["win"])
    gd = ssd.linear_bwd(g["ddt"], y, p["wdt"])
    gb = ssd.linear_bwd(g["dbeta"], y, p["wb"], pre=pre, activation="sigmoid", bias=True)
    gn = ssd.layer_norm_bwd(gi["dx"] + gd["dx"] + gb["dx"], s, st, p["nw"], bias=True, d_sum=dout)
    return dict(wout=go["dweight"], A=g["dA"], dt_bias=g["ddt_bias"], win=gi["dweight"],
                wdt=gd["dweight"], wb=gb["dweight"], bb=gb["dbias"], nw=gn["dweight"],
                nb=gn["dbias"], x=gn["dx"], init=g["d_init"])


def _autograd(p, x, res, init, dout):
    """The block in fp64 on the CPU, token by token, and its gradients."""
    torch = torch_mod()
    q = {k: v.double().cpu().requires_grad_(True) for k, v in p.items()}
    xx = x.double().cpu().requires_grad_(True)
    S = ini = init.double().cpu().requires_grad_(True)
    s = xx + res.double().cpu()
    y = torch.nn.functional.layer_norm(s, (s.shape[-1],), q["nw"], q["nb"], 1e-5)
    qq, kk, v = _split(y @ q["win"].t())
    unit = lambda t: (t / torch.sqrt((t * t).sum(-1, keepdim=True) + 1e-6)  # noqa: E731
                      ).repeat_interleave(H // G, -2)
    qq, kk = unit(qq), unit(kk)
    keep = torch.exp(q["A"] * torch.nn.functional.softplus(y @ q["wdt"].t() + q["dt_bias"]))
    beta = torch.sigmoid(y @ q["wb"].t() + q["bb"])
    os = []
    for t in range(s.shape[1]):
        P0 = keep[:, t, :, None, None] * S
        u = beta[:, t, :, None] * (v[:, t] - (P0 * kk[:, t, :, :, None]).sum(2))
        S = P0 + kk[:, t, :, :, None] * u[:, :, None, :]
        os.append((S * qq[:, t, :, :, None]).sum(2) / math.sqrt(N))
    out = torch.stack(os, 1).flatten(2) @ q["wout"].t() + s
    out.backward(dout.double().cpu())
    return out.detach(), S.detach(), dict({k: v.grad for k, v in q.items()}, x=xx.grad, init=ini.grad)


def test_block_gradient_against_autograd_in_64_bits():
    """fp32 against autograd through the definition.  A value is off by at most
    2^-18 of the largest terms behind it (the products and the scan both), about
    ten such steps follow each other, and a gradient's norm is at least a
    hundredth of its terms': 10 * 2^-18 * 100 < 4e-3."""
    import mamba_ssd_chunked_chunk_amd as ssd
    p, t = _block(81, 48, "f32")
    x, res, dout = t(2, 150, 48), t(2, 150, 48), t(2, 150, 48)
    init = t(2, H, N, P, std=0.3)
    out, fin, saved = _forward(ssd, p, x, res, init)
    g = _backward(ssd, p, saved, init, dout)
    want, S, ref = _autograd(p, x, res, init, dout)
    assert float((out.double().cpu() - want).norm() / want.norm()) < 1e-5
    assert float((fin.double().cpu() - S).norm() / S.norm()) < 1e-4
    assert set(g) == set(ref)
    for k, r in ref.items():
        rel = float((g[k].double().cpu() - r).norm() / r.norm())
        log("block gradient", k, "%.2e" % rel)
        assert rel < 4e-3, (k, rel)


def test_block_gradient_bf16_against_fp32():
    """The block in bf16 against itself in fp32 on the same values.  Ten roundings
    of 2^-8 in a row, each of which a product may carry on threefold: 0.12."""
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    p, t = _block(82, 64, "bf16")
    x, res, dout = t(2, 200, 64), t(2, 200, 64), t(2, 200, 64)
    init = t(2, H, N, P, std=0.3, dtype=torch.float32)
    wide = {k: v.float() for k, v in p.items()}
    _, fin, saved = _forward(ssd, p, x, res, init)
    g = _backward(ssd, p, saved, init, dout)
    _, fin32, saved = _forward(ssd, wide, x.float(), res.float(), init)
    g32 = _backward(ssd, wide, saved, init, dout.float())
    for k, r in dict(g32, fin=fin32).items():
        got = fin if k == "fin" else g[k]
        rel = float((got.float() - r).norm() / r.norm())
        log("bf16 block", k, "%.2e" % rel)
        assert rel < 0.12, (k, rel)


def test_block_token_by_token():
    """A prompt, then steps, against one pass over all tokens (fp32)."""
    import mamba_ssd_chunked_chunk_amd as ssd
    p, t = _block(83, 48, "f32")
    x, res, init = t(2, 100, 48), t(2, 100, 48), t(2, H, N, P, std=0.3)
    whole, fin, _ = _forward(ssd, p, x, res, init)
    _, state, _ = _forward(ssd, p, x[:, :70].contiguous(), res[:, :70].contiguous(), init)
    for i in range(70, 100):
        _, s, _, (q, k, v), dt, beta, _ = _front(ssd, p, x[:, i].contiguous(), res[:, i].contiguous())
        o = ssd.delta_step(state, q, k, v, dt, p["A"], beta, dt_bias=p["dt_bias"], normalize=True)
        out = ssd.linear(o.reshape(2, H * P), p["wout"], residual=s)
        assert float((out - whole[:, i]).norm() / whole[:, i].norm()) < 1e-5, i
    assert float((state - fin).norm() / fin.norm()) < 1e-4


def test_block_from_a_graph():
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    p, t = _block(84, 64, "bf16")
    x, res, dout = t(2, 130, 64), t(2, 130, 64), t(2, 130, 64)
    init = t(2, H, N, P, std=0.3, dtype=torch.float32)

    def work():
        out, fin, saved = _forward(ssd, p, x, res, init)
        g = _backward(ssd, p, saved, init, dout)
        return [out, fin] + [g[k] for k in sorted(g)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work()
    for i in range(3):
        for buf in (x, res, dout):
            buf.copy_(torch.randn_like(buf))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for a, b in zip(got, work()):
            assert torch.equal(a, b)
