"""The linear layer and the gated recurrence as they are used together: a
recurrent block (gates and input from one product each, the recurrence, the
projection with the residual), its gradient, its decode steps, and its replay
from a graph; and the Mamba-2 mixer between two linear layers."""
import math

import numpy as np
import pytest

from gpu_util import log, to_f64, torch_mod

pytestmark = pytest.mark.gpu


def _block(seed, dm, d, io):
    torch = torch_mod()
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    rng = np.random.default_rng(seed)

    def t(*shape, std=1.0, dtype=dt):
        return torch.from_numpy((rng.normal(size=shape) * std).astype(np.float32)).to("cuda").to(dtype)
    a = 0.9 + 0.0995 * rng.random(d)
    return dict(win=t(d, dm, std=dm ** -0.5), wg=t(2 * d, dm, std=dm ** -0.5),
                bg=t(2 * d, std=0.5, dtype=torch.float32), wout=t(dm, d, std=d ** -0.5),
                lam=torch.from_numpy(np.log(np.expm1(-np.log(a) / 8)).astype(np.float32)).to("cuda")), t


def _forward(ssd, p, u, init=None, keep=False):
    x, pre = ssd.linear(u, p["win"], activation="gelu", return_pre=True)
    gates = ssd.linear(u, p["wg"], bias=p["bg"])
    y, fin, st = ssd.gated_scan(x, gates, p["lam"], initial_state=init, return_final_state=True,
                                return_states=True)
    out = ssd.linear(y, p["wout"], residual=u)
    return (out, fin, (x, pre, gates, y, st)) if keep else (out, fin)


def _backward(ssd, p, u, saved, dout):
    x, pre, gates, y, st = saved
    go = ssd.linear_bwd(dout, y, p["wout"])
    gs = ssd.gated_scan_bwd(x, gates, p["lam"], go["dx"], states=st)
    gg = ssd.linear_bwd(gs["dgates"], u, p["wg"], bias=True)
    gi = ssd.linear_bwd(gs["dx"], u, p["win"], pre=pre, activation="gelu")
    return dict(wout=go["dweight"], lam=gs["dlam"], wg=gg["dweight"], bg=gg["dbias"],
                win=gi["dweight"], u=(dout + gg["dx"] + gi["dx"]))


def test_block_gradient_against_autograd_in_64_bits():
    """The block's gradient in fp32 against autograd through the definition in
    fp64 on the CPU.  Each of the block's values is off by at most about 2^-18
    of the largest terms behind it; ten such steps follow each other, and a
    gradient's norm is at least a hundredth of its terms': 10 * 2^-18 * 100
    < 4e-3 of the norm."""
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    p, t = _block(61, 48, 40, "f32")
    u, dout = t(2, 150, 48), t(2, 150, 48)
    out, fin, saved = _forward(ssd, p, u, keep=True)
    g = _backward(ssd, p, u, saved, dout)
    torch.cuda.synchronize()
    q = {k: v.double().cpu().requires_grad_(True) for k, v in p.items()}
    uu = u.double().cpu().requires_grad_(True)
    x = torch.nn.functional.gelu(uu @ q["win"].t())
    z = uu @ q["wg"].t() + q["bg"]
    rate = 8 * torch.nn.functional.softplus(q["lam"]) * torch.sigmoid(z[..., :40])
    a, add = torch.exp(-rate), torch.sqrt(-torch.expm1(-2 * rate)) * torch.sigmoid(z[..., 40:]) * x
    h, hs = torch.zeros(2, 40, dtype=torch.float64), []
    for k in range(150):
        h = a[:, k] * h + add[:, k]
        hs.append(h)
    want = torch.stack(hs, 1) @ q["wout"].t() + uu
    want.backward(dout.double().cpu())
    w = want.detach()
    assert float((out.double().cpu() - w).norm() / w.norm()) < 1e-5
    for k, ref in dict(q, u=uu).items():
        r = ref.grad
        rel = float((g[k].double().cpu() - r).norm() / r.norm())
        log("block gradient", k, "%.2e" % rel)
        assert rel < 4e-3, (k, rel)


def test_decode_continues_the_prompt():
    """Step by step after a prompt gives the whole pass: bf16, each layer's
    output off by one rounding (2^-8 of its value) of the same fp32 values; the
    rows' products sum K terms of both, so the norm of the difference stays
    below 4 roundings."""
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    p, t = _block(62, 96, 130, "bf16")
    u = t(3, 90, 96)
    whole, fin = _forward(ssd, p, u)
    out, state = _forward(ssd, p, u[:, :80].contiguous())
    for k in range(80, 90):
        v = u[:, k].contiguous()
        y = ssd.gated_step(state, ssd.linear(v, p["win"], activation="gelu"),
                           ssd.linear(v, p["wg"], bias=p["bg"]), p["lam"])
        o = ssd.linear(y, p["wout"], residual=v)
        torch.cuda.synchronize()
        d = to_f64(o) - to_f64(whole[:, k])
        assert np.linalg.norm(d) <= 4 * 2.0 ** -8 * np.linalg.norm(to_f64(whole[:, k]))
    d = to_f64(state) - to_f64(fin)
    assert np.linalg.norm(d) <= 4 * 2.0 ** -8 * np.linalg.norm(to_f64(fin))


@pytest.mark.parametrize("l", [1, 700])
def test_graph_replays_equal_eager(l):
    """Forward, gradient and a step captured in one graph; every replay, with
    new inputs and eager work between, equals the eager calls bit for bit."""
    import mamba_ssd_chunked_chunk_amd as ssd
    torch = torch_mod()
    p, t = _block(63, 264, 72, "bf16")
    u, dout, h = t(2, l, 264), t(2, l, 264), t(2, 72, dtype=torch.float32)

    def work(st):
        out, fin, saved = _forward(ssd, p, u, keep=True)
        g = _backward(ssd, p, u, saved, dout)
        y = ssd.gated_step(st, saved[0][:, -1].contiguous(), saved[2][:, -1].contiguous(), p["lam"])
        return [out, fin, y] + [g[k] for k in sorted(g)]

    state = h.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work(state)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work(state)
    for k in range(4):
        u.copy_(t(2, l, 264))
        state.copy_(h)
        torch.cuda.synchronize()
        eager = h.clone()
        want = [v.clone() for v in work(eager)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), k
        assert torch.equal(state, eager)


def test_mixer_between_its_projections():
    """A Mamba-2 block in the library's calls: z, x|B|C and dt from three
    products of one weight's rows, the mixer, and the output projection with
    the residual, against the same block from the oracle's parts."""
    import mamba_ssd_chunked_chunk_amd as ssd
    import oracle
    from oracle import neighbors as nb
    torch = torch_mod()
    b, l, dm, h, p, n, g = 2, 70, 128, 4, 32, 32, 1
    ch = h * p + 2 * g * n
    rng = np.random.default_rng(64)

    def t(*shape, std=1.0):
        return torch.from_numpy((rng.normal(size=shape) * std).astype(np.float32)).to("cuda")
    u, win = t(b, l, dm), t(h * p + ch + h, dm, std=dm ** -0.5)
    wout, cw, cb = t(dm, h * p, std=(h * p) ** -0.5), t(ch, 4, std=0.4), t(ch, std=0.1)
    A, D, bias, nw = -torch.exp(t(h)), t(h), t(h, std=0.2), 1 + 0.1 * t(h * p)
    cut = [0, h * p, h * p + ch, h * p + ch + h]
    z, xbc, dt = (ssd.linear(u, win[i:j]) for i, j in zip(cut, cut[1:]))
    y = ssd.mixer_forward(xbc, dt, A, cw, h, p, n, g, z=z, conv_bias=cb, D=D, dt_bias=bias,
                          norm_weight=nw, chunk_size=32)
    out = ssd.linear(y.view(b, l, h * p), wout, residual=u)
    torch.cuda.synchronize()
    f = lambda v: v.cpu().numpy()  # noqa: E731
    proj = to_f64(u) @ to_f64(win).T
    zo, xo, dto = (proj[..., i:j].astype(np.float32) for i, j in zip(cut, cut[1:]))
    x, B, C, _ = nb.conv1d_silu(xo, f(cw), h, p, n, g, bias=f(cb))
    ys, _ = oracle.scan(x.astype(np.float32), dto, f(A), B.astype(np.float32),
                        C.astype(np.float32), f(D), f(bias), io="f32")
    yo = nb.gated_norm(ys.reshape(b * l, h * p).astype(np.float32), zo.reshape(b * l, h * p),
                       f(nw), h * p, 1e-5)
    want = yo.reshape(b, l, h * p) @ to_f64(wout).T + to_f64(u)
    d = to_f64(out) - want
    # fp32 io throughout: the scan's own bar is 1e-4 of its values
    assert np.linalg.norm(d) <= 2e-4 * np.linalg.norm(want)
    assert math.isfinite(float(np.abs(d).max()))
