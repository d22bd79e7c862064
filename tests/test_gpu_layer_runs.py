"""The layer operators used as a program uses them: a layer's prompt, single tokens and gradients run
together, captured graphs, other streams, tokens that belong to no sequence, offsets past 32 bits."""
import ctypes

import pytest
import torch

import state_space_sequence_mamba3_amd as m3
from tests import layer_ref as R
from tests.gpu_util import device, note
from tests.test_gpu_layer import BF16, F32, dev, gen, rand, scan_inputs, up

pytestmark = pytest.mark.gpu

D, N, RANK, M, W, EPS = 48, 16, 5, 40, 4, 1e-5   # channels, states, rank of dt, model width, taps


def layer_weights(g):
    return dict(norm=rand(g, M) * 0.1 + 1, win=rand(g, M, 2 * D, std=M ** -0.5), conv=rand(g, D, W, std=0.5),
                cbias=rand(g, D, std=0.1), wx=rand(g, D, RANK + 2 * N, std=D ** -0.5), wdt=rand(g, RANK, D, std=0.4),
                dtb=rand(g, D) - 2, A=-torch.exp(rand(g, D, N, std=0.3)), skip=rand(g, D), wout=rand(g, D, M, std=D ** -0.5))


def layer_plain(p, h, res):
    """One layer in plain torch (any type, differentiable): the layer's output and its residual stream."""
    s = h + res
    v = s * torch.rsqrt((s * s).mean(-1, keepdim=True) + EPS) * p["norm"]
    x, z = (v @ p["win"]).split([D, D], -1)
    pad = torch.cat([x.new_zeros(x.shape[0], W - 1, D), x], 1)
    c = sum(pad[:, j:j + x.shape[1]] * p["conv"][:, j] for j in range(W)) + p["cbias"]
    x = c * torch.sigmoid(c)
    r, B, C = (x @ p["wx"]).split([RANK, N, N], -1)
    step = torch.nn.functional.softplus(r @ p["wdt"] + p["dtb"])
    state, ys = x.new_zeros(x.shape[0], D, N), []
    for t in range(x.shape[1]):
        state = torch.exp(step[:, t, :, None] * p["A"]) * state + (step[:, t] * x[:, t])[..., None] * B[:, t, None]
        ys.append((state * C[:, t, None]).sum(-1) + p["skip"] * x[:, t])
    y = torch.stack(ys, 1) * z * torch.sigmoid(z)
    return y @ p["wout"], s


def layer_prompt(p, h, res):
    """The same by the library: outputs, residual stream, states after the prompt, and what a backward needs."""
    n = m3.mamba3_rmsnorm_fwd(h, p["norm"], residual=res, eps=EPS)
    xz = n["y"] @ p["win"]
    x, z = xz[:, :, :D], xz[:, :, D:]
    xc, conv = m3.mamba3_conv_fwd(x, p["conv"], p["cbias"])
    proj = xc @ p["wx"]
    dt = proj[:, :, :RANK] @ p["wdt"]
    B, C = proj[:, :, RANK:RANK + N].unflatten(2, (1, N)), proj[:, :, RANK + N:].unflatten(2, (1, N))
    y, state = m3.mamba3_selective_scan_fwd(xc, dt, p["A"], B, C, p["skip"], z=z, dt_bias=p["dtb"], dt_softplus=True)
    return y @ p["wout"], n["residual"], conv, state, (n["y"], x, z, xc, dt, B, C, proj, y)


def layer_token(p, h, res, conv, state):
    n = m3.mamba3_rmsnorm_fwd(h, p["norm"], residual=res, eps=EPS)
    x, z = (n["y"] @ p["win"]).split([D, D], -1)
    xc = m3.mamba3_conv_step(x, p["conv"], p["cbias"], conv=conv)
    r, B, C = (xc @ p["wx"]).split([RANK, N, N], -1)
    y = m3.mamba3_selective_step(xc, r @ p["wdt"], p["A"], B.unflatten(1, (1, N)), C.unflatten(1, (1, N)), p["skip"],
                                 h=state, z=z, dt_bias=p["dtb"], dt_softplus=True)
    return y @ p["wout"], n["residual"]


def near(got, want, what):
    """Each operator is held to its own bound by its own tests; over the chain of five operators and four
    products of up to 96 terms fp32's roundings (2^-24 each, a few hundred in a row, none amplified
    by more than the products' condition) stay below 1e-4 of the largest value."""
    got, want = got.detach().cpu().double(), want.detach().double()
    err = float((got - want).abs().max() / want.abs().max())
    assert err < 1e-4, (what, err)


def test_layer_prompt_then_tokens():
    g = gen(1)
    p, b, L, n = layer_weights(g), 3, 41, 33
    h, res = rand(g, b, L, M), rand(g, b, L, M)
    want, stream = layer_plain({k: v.double() for k, v in p.items()}, h.double(), res.double())
    q = dev(p)
    out, rs, conv, state, _ = layer_prompt(q, up(h[:, :n]), up(res[:, :n]))
    near(out, want[:, :n], "prompt")
    near(rs, stream[:, :n], "residual")
    for t in range(n, L):
        o, rs = layer_token(q, up(h[:, t]), up(res[:, t]), conv, state)
        near(o, want[:, t], f"token {t}")
        near(rs, stream[:, t], f"residual {t}")


def test_layer_gradients():
    """The operators' backward passes chained by hand against autograd through the plain layer in 64 bits."""
    g = gen(2)
    p, b, L = layer_weights(g), 2, 37
    h, res, dout, dstream = rand(g, b, L, M), rand(g, b, L, M), rand(g, b, L, M), rand(g, b, L, M)
    leaf = {k: v.double().requires_grad_() for k, v in {**p, "h": h, "res": res}.items()}
    out, stream = layer_plain({k: leaf[k] for k in p}, leaf["h"], leaf["res"])
    torch.autograd.backward([out, stream], [dout.double(), dstream.double()])
    q = dev(p)
    _, s, _, _, (nrm, x, z, xc, dt, B, C, proj, y) = layer_prompt(q, up(h), up(res))
    do = up(dout)
    gr = {"wout": y.flatten(0, 1).t() @ do.flatten(0, 1)}
    sc = m3.mamba3_selective_scan_bwd(xc, dt, q["A"], B, C, q["skip"], z=z, dt_bias=q["dtb"], dt_softplus=True,
                                      dy=do @ q["wout"].t())
    gr.update(A=sc["dA"], skip=sc["dD"], dtb=sc["ddt_bias"], wdt=proj[:, :, :RANK].flatten(0, 1).t() @ sc["ddt"].flatten(0, 1))
    dproj = torch.cat([sc["ddt"] @ q["wdt"].t(), sc["dB"].flatten(2), sc["dC"].flatten(2)], -1)
    gr["wx"] = xc.flatten(0, 1).t() @ dproj.flatten(0, 1)
    cv = m3.mamba3_conv_bwd(x, q["conv"], q["cbias"], dy=sc["dx"] + dproj @ q["wx"].t())
    gr.update(conv=cv["dweight"], cbias=cv["dbias"])
    dxz = torch.cat([cv["dx"], sc["dz"]], -1)
    gr["win"] = nrm.flatten(0, 1).t() @ dxz.flatten(0, 1)
    nb = m3.mamba3_rmsnorm_bwd(s, q["norm"], dy=dxz @ q["win"].t(), dresidual_out=up(dstream), eps=EPS)
    gr.update(norm=nb["dweight"], h=nb["dx"], res=nb["dresidual"])
    assert set(gr) == set(leaf)
    for k in gr:
        near(gr[k], leaf[k].grad, k)


# ----------------------------------------------------------------------------- calls of every kind, for the tests below
def calls(g, dtype):
    """name -> (inputs, function of them that returns tensors)."""
    out = {}
    for tag, (b, L, cu) in dict(padded=(2, 150, None), packed=(1, 260, [0, 7, 7, 200, 260])).items():
        S = len(cu) - 1 if cu else b
        cut = dict(cu=torch.tensor(cu, dtype=torch.int32)) if cu else {}
        x = rand(g, b, L, 72, dtype=dtype)
        conv = dict(x=x, w=rand(g, 72, 4), bias=rand(g, 72), cin=rand(g, S, 3, 72, dtype=dtype), dy=rand(g, *x.shape, dtype=dtype),
                    dco=rand(g, S, 3, 72, dtype=dtype), **cut)
        out[f"conv {tag}"] = (conv, lambda v: m3.mamba3_conv_fwd(v["x"], v["w"], v["bias"], conv_in=v["cin"], cu_seqlens=v.get("cu")))
        out[f"conv_bwd {tag}"] = (conv, lambda v: m3.mamba3_conv_bwd(v["x"], v["w"], v["bias"], dy=v["dy"], dconv_out=v["dco"],
                                                                    conv_in=v["cin"], cu_seqlens=v.get("cu")).values())
        a, kw, dy, dho, c = scan_inputs((b, L, 40, 16, 1, cu), dtype, True)
        sc = {**a, **kw, "dy": dy, "dho": dho, **({"cu": c} if cu else {})}
        args = ("x", "dt", "A", "B", "C", "D")
        opts = ("z", "dt_bias", "dt_softplus", "h_in")
        out[f"scan {tag}"] = (sc, lambda v: m3.mamba3_selective_scan_fwd(*[v[k] for k in args], **{k: v[k] for k in opts},
                                                                        cu_seqlens=v.get("cu")))
        out[f"scan_bwd {tag}"] = (sc, lambda v: m3.mamba3_selective_scan_bwd(*[v[k] for k in args], **{k: v[k] for k in opts},
                                                                            dy=v["dy"], dh_out=v["dho"],
                                                                            cu_seqlens=v.get("cu")).values())
    nm = dict(x=rand(g, 50, 256, dtype=dtype), res=rand(g, 50, 256), w=rand(g, 256), dy=rand(g, 50, 256, dtype=dtype))
    out["norm"] = (nm, lambda v: [t.view(torch.uint8) for t in m3.mamba3_rmsnorm_fwd(v["x"], v["w"], residual=v["res"],
                                                                                    quant="e4m3").values()])
    out["norm_bwd"] = (nm, lambda v: m3.mamba3_rmsnorm_bwd(v["res"], v["w"], dy=v["dy"], dresidual_out=v["res"]).values())
    # the steps return the state they leave, from a copy of the one they start with
    st = dict(x=rand(g, 5, 72, dtype=dtype), w=rand(g, 72, 4), conv=rand(g, 9, 3, 72, dtype=dtype),
              slots=torch.tensor([3, -1, 8, 0, 9], dtype=torch.int32))

    def conv_step(v):
        conv, y = v["conv"].clone(), torch.zeros_like(v["x"])
        return m3.mamba3_conv_step(v["x"], v["w"], conv=conv, slots=v["slots"], y=y), conv

    out["conv_step"] = (st, conv_step)
    ss = dict(x=rand(g, 5, 40, dtype=dtype), dt=rand(g, 5, 40, dtype=dtype), A=-torch.exp(rand(g, 40, 16)),
              B=rand(g, 5, 2, 16, dtype=dtype), C=rand(g, 5, 2, 16, dtype=dtype), h=rand(g, 9, 40, 16), slots=st["slots"])

    def scan_step(v):
        h, y = v["h"].clone(), torch.zeros_like(v["x"])
        return m3.mamba3_selective_step(v["x"], v["dt"], v["A"], v["B"], v["C"], h=h, dt_softplus=True, slots=v["slots"], y=y), h

    out["scan_step"] = (ss, scan_step)
    return out


NAMES = [f"{k} {t}" for k in ("conv", "conv_bwd", "scan", "scan_bwd") for t in ("padded", "packed")] + \
    ["norm", "norm_bwd", "conv_step", "scan_step"]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("name", NAMES)
def test_captured_and_replayed(name, dtype):
    """A captured call replayed on new inputs, with eager work between the replays, equals the eager call
    bit for bit; two graphs of one call are replayed in turn."""
    note(f"graph of {name} {dtype}")
    inp, f = calls(gen(3), dtype)[name]
    v = dev(inp)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        f(v)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs = list(f(v))
        graphs.append((gr, outs))
    for k in range(3):
        for key, t in v.items():       # other inputs: the channels of the first ones rolled
            if isinstance(t, torch.Tensor) and t.is_floating_point():
                t.copy_(t.roll(1, 0 if t.dim() == 1 else -1 if key not in ("A", "w") else 0))
        want = [t.clone() for t in f(v)]
        for gr, outs in graphs:
            gr.replay()
            torch.cuda.synchronize()
            for a, b in zip(outs, want):
                assert torch.equal(a, b), (name, k)
            for t in outs:
                t.zero_()


@pytest.mark.parametrize("name", NAMES)
def test_on_another_stream(name):
    """The current stream of the call, and calls on two streams at once: the same bits."""
    inp, f = calls(gen(4), BF16)[name]
    v = dev(inp)
    want = [t.clone() for t in f(v)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append([t.clone() for t in f(v)])
    torch.cuda.synchronize()
    for o in got:
        assert all(torch.equal(a, b) for a, b in zip(o, want))


def test_stream_argument():
    g = gen(5)
    x, w = up(rand(g, 2, 50, 64)), up(rand(g, 64, 4))
    want, _ = m3.mamba3_conv_fwd(x, w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    a, _ = m3.mamba3_conv_fwd(x, w, stream=s)
    b, _ = m3.mamba3_conv_fwd(x, w, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)


# ----------------------------------------------------------------------------- tokens of no sequence
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cu", [[3, 10, 10, 25], [0, 7, 9, 9], [40, 40, 40, 40], [5, 5, 38, 39]])
def test_tokens_outside_the_sequences(cu, dtype):
    """Tokens before the first and behind the last sequence: no part in any result, their rows untouched."""
    T, C, S = 40, 24, 3
    g = gen(sum(cu))
    note(f"tokens outside {cu} {dtype}")
    cut, lo, hi = torch.tensor(cu, dtype=torch.int32), cu[0], cu[-1]
    out = torch.ones(T, dtype=torch.bool)
    out[lo:hi] = False
    x, w, bias, cin = rand(g, 1, T, C, dtype=dtype), rand(g, C, 4), rand(g, C), rand(g, S, 3, C, dtype=dtype)
    dy, dco = rand(g, 1, T, C, dtype=dtype), rand(g, S, 3, C, dtype=dtype)
    x[0, out], dy[0, out] = float("nan"), float("nan")

    def inside(t):
        t = t.clone()
        t[0, out] = 0
        return t

    def untouched(t, what):
        assert bool((t[0, out.to(device())] == 7).all()), what
        return inside(t.cpu())

    y = torch.full((1, T, C), 7.0, dtype=dtype, device=device())
    _, co = m3.mamba3_conv_fwd(up(x), up(w), up(bias), conv_in=up(cin), cu_seqlens=up(cut), y=y)
    ref, mag = (R.conv(inside(x), w, bias, True, cin, cu, inside(dy), dco, mag=m) for m in (False, True))
    R.check(untouched(y, "y"), ref["y"], mag["y"], 20, "y")
    assert torch.equal(co.cpu().double(), ref["conv_out"])
    dx = torch.full((1, T, C), 7.0, dtype=dtype, device=device())
    dw, db = torch.empty(C, 4, device=device()), torch.empty(C, device=device())
    dci, ws = torch.empty(S, 3, C, dtype=dtype, device=device()), torch.empty(1 << 20, dtype=torch.uint8, device=device())
    keep = [up(t) for t in (x, w, bias, cin, cut, dy, dco)]
    xp, wp, bp, cp, up_, yp, op = (t.data_ptr() for t in keep)
    code = m3.MAMBA3_BF16 if dtype == BF16 else m3.MAMBA3_F32
    a = m3.ConvBwdArgs(m3.ConvArgs(1, T, C, 4, code, 1, up_, S, 0, xp, wp, bp, cp, None, None), 0, yp, op, dx.data_ptr(),
                       dw.data_ptr(), db.data_ptr(), dci.data_ptr(), ws.data_ptr(), ws.numel())
    assert m3.lib().mamba3_conv_bwd(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == m3.MAMBA3_OK
    torch.cuda.synchronize()
    R.check(untouched(dx, "dx"), ref["dx"], mag["dx"], 40, "dx")
    for got, k in ((dw, "dweight"), (db, "dbias"), (dci, "dconv_in")):
        R.check(got, ref[k], mag[k], T + 40, k)

    a, kw, dy, dho, _ = scan_inputs((1, T, C, 16, 1, cu), dtype, True)
    full = {**a, **kw}
    toks = ("x", "dt", "B", "C", "z")
    bad = {k: full[k].clone() for k in toks}
    for k in toks:
        bad[k][0, out] = float("nan")
        full[k] = inside(full[k])
    dyb = dy.clone()
    dyb[0, out] = float("nan")
    ref, mag = (R.scan(full["x"], full["dt"], full["A"], full["B"], full["C"], full["D"], full["z"], full["dt_bias"], True,
                       full["h_in"], cu, inside(dy), dho, mag=m) for m in (False, True))
    q = dev({**full, **bad})
    y = torch.full((1, T, C), 7.0, dtype=dtype, device=device())
    _, h = m3.mamba3_selective_scan_fwd(*[q[k] for k in ("x", "dt", "A", "B", "C", "D")], z=q["z"], dt_bias=q["dt_bias"],
                                        dt_softplus=True, h_in=q["h_in"], cu_seqlens=up(cut), y=y)
    R.check(untouched(y, "y"), ref["y"], mag["y"], 70 * T + 48, "scan y")
    R.check(h, ref["h_out"], mag["h_out"], 70 * T + 16, "h_out")
    o = {k: torch.full(s, 7.0, dtype=dtype, device=device()) for k, s in
         dict(dx=(1, T, C), ddt=(1, T, C), dB=(1, T, 1, 16), dC=(1, T, 1, 16), dz=(1, T, C)).items()}
    f = {k: torch.empty(s, device=device()) for k, s in dict(dA=(C, 16), dD=(C,), ddt_bias=(C,), dh_in=(S, C, 16)).items()}
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=device())
    dyd, dhod = up(dyb), up(dho)
    p = {k: t.data_ptr() for k, t in q.items() if isinstance(t, torch.Tensor)}
    fa = m3.SelectiveScanArgs(1, T, C, 16, 1, code, 1, keep[4].data_ptr(), S, 0, 0, 0, 0, 0, p["x"], p["dt"], p["B"], p["C"],
                              p["z"], p["A"], p["D"], p["dt_bias"], p["h_in"], None, None, None, 0)
    ba = m3.SelectiveScanBwdArgs(fa, 0, dyd.data_ptr(), dhod.data_ptr(),
                                 *[o[k].data_ptr() for k in ("dx", "ddt", "dB", "dC", "dz")],
                                 *[f[k].data_ptr() for k in ("dA", "dD", "ddt_bias", "dh_in")], ws.data_ptr(), ws.numel())
    assert m3.lib().mamba3_selective_scan_bwd(ctypes.byref(ba), torch.cuda.current_stream().cuda_stream) == m3.MAMBA3_OK
    torch.cuda.synchronize()
    for k, t in o.items():
        R.check(untouched(t, k), ref[k], mag[k], 140 * T + 112, k)
    for k, t in f.items():
        R.check(t, ref[k], mag[k], 140 * T + 112, k)


# ----------------------------------------------------------------------------- offsets past 32 bits
def test_rows_far_apart():
    """Token rows whose last elements lie more than 2^32 bytes behind the first: the same bits as dense rows."""
    row, T, C, n = 1 << 25, 80, 40, 16
    wide = torch.empty(T * row, dtype=BF16, device=device())
    view = torch.as_strided(wide, (1, T, C + 2 * n), (T * row, row, 1), 8)
    g = gen(6)
    note(f"rows {row} apart: {wide.numel() * 2 >> 20} MiB")
    view.copy_(up(rand(g, 1, T, C + 2 * n, dtype=BF16)))
    x, B, C_ = view[:, :, :C], view[:, :, C:C + n].unflatten(2, (1, n)), view[:, :, C + n:].unflatten(2, (1, n))
    w, A = up(rand(g, C, 4)), up(-torch.exp(rand(g, C, n)))
    d = [t.contiguous() for t in (x, B, C_)]
    assert torch.equal(m3.mamba3_conv_fwd(x, w)[0], m3.mamba3_conv_fwd(d[0], w)[0])
    a, b = (m3.mamba3_conv_bwd(t, w, dy=t) for t in (x, d[0]))
    assert all(torch.equal(a[k], b[k]) for k in a)
    a = m3.mamba3_selective_scan_fwd(x, x, A, B, C_, z=x, dt_softplus=True)
    b = m3.mamba3_selective_scan_fwd(d[0], d[0], A, d[1], d[2], z=d[0], dt_softplus=True)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    a = m3.mamba3_selective_scan_bwd(x, x, A, B, C_, z=x, dt_softplus=True, dy=x)
    b = m3.mamba3_selective_scan_bwd(d[0], d[0], A, d[1], d[2], z=d[0], dt_softplus=True, dy=d[0])
    assert all(torch.equal(a[k], b[k]) for k in a)
    a, b = (m3.mamba3_rmsnorm_fwd(t[0])["y"] for t in (x, d[0]))
    assert torch.equal(a, b)
    st = up(rand(g, T, C, n))
    a = m3.mamba3_selective_step(x[0], x[0], A, B[0], C_[0], h=st.clone(), dt_softplus=True)
    b = m3.mamba3_selective_step(d[0][0], d[0][0], A, d[1][0], d[2][0], h=st.clone(), dt_softplus=True)
    assert torch.equal(a, b)


def test_binding_refusals_on_the_device():
    x, w = torch.zeros(2, 6, 8, device=device()), torch.zeros(8, 4, device=device())
    bad = [lambda: m3.mamba3_conv_fwd(x, w.cpu()), lambda: m3.mamba3_conv_fwd(x, w.t()), lambda: m3.mamba3_conv_fwd(x, w[:4]),
           lambda: m3.mamba3_conv_fwd(x[:, :5], w), lambda: m3.mamba3_conv_fwd(x.transpose(0, 1), w),
           lambda: m3.mamba3_conv_fwd(x, w, cu_seqlens=torch.tensor([0, 6], dtype=torch.int32, device=device())),
           lambda: m3.mamba3_conv_step(x[:, 0], w, conv=torch.zeros(2, 4, 8, device=device())),
           lambda: m3.mamba3_rmsnorm_fwd(x, quant="e5m2"), lambda: m3.mamba3_rmsnorm_fwd(x, want_y=False),
           lambda: m3.mamba3_rmsnorm_fwd(x, residual=x[:1])]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    # every second of six tokens is a valid view: one distance of 16 within and across the sequences
    assert torch.equal(m3.mamba3_conv_fwd(x[:, ::2], w)[0], m3.mamba3_conv_fwd(x[:, ::2].contiguous(), w)[0])
    for f in (lambda: m3.mamba3_conv_fwd(x.half(), w.half()), lambda: m3.mamba3_conv_fwd(x, w.bfloat16()),
              lambda: m3.mamba3_rmsnorm_fwd(x, residual=x.half())):
        with pytest.raises(TypeError):
            f()
    for f in (lambda: m3.mamba3_conv_fwd(x, torch.zeros(8, 9, device=device())), lambda: m3.mamba3_rmsnorm_fwd(x, quant="int8",
                                                                                                               qblock=5),
              lambda: m3.mamba3_conv_fwd(x, w, y=x), lambda: m3.mamba3_rmsnorm_fwd(x, eps=-1.0)):
        with pytest.raises(m3.Mamba3Error):
            f()
