"""The gated layer's operators used as a program uses them: a layer's prompt, single tokens, states put aside and
taken back, and gradients; captured graphs, several streams at once; arrays past 32 bits."""
import pytest
import torch

import state_space_sequence_mamba3_amd as m3
from tests import gated_ref as R
from tests.gpu_util import device, note
from tests.test_gpu_layer import BF16, F32, dev, gen, rand, up

pytestmark = pytest.mark.gpu

M, D, G, W, EPS = 40, 96, 6, 4, 1e-5      # model width, channels, groups of the norm, taps


def layer_weights(g):
    return dict(win=rand(g, M, 4 * D, std=M ** -0.5), conv=rand(g, D, W, std=0.5), cbias=rand(g, D, std=0.1), decay=rand(g, D) - 4,
                gn=rand(g, D) * 0.1 + 1, gb=rand(g, D, std=0.1), wout=rand(g, D, M, std=D ** -0.5))


def layer_plain(p, h):
    """One layer in plain torch (any type, differentiable)."""
    x, gate, i, z = (h @ p["win"]).split([D] * 4, -1)
    pad = torch.cat([x.new_zeros(x.shape[0], W - 1, D), x], 1)
    c = sum(pad[:, j:j + x.shape[1]] * p["conv"][:, j] for j in range(W)) + p["cbias"]
    x = c * torch.sigmoid(c)
    la = -8.0 * torch.nn.functional.softplus(p["decay"]) * torch.sigmoid(gate)
    u = torch.sqrt(-torch.expm1(2 * la)) * torch.sigmoid(i) * x
    state, ys = x.new_zeros(x.shape[0], D), []
    for t in range(x.shape[1]):
        state = torch.exp(la[:, t]) * state + u[:, t]
        ys.append(state)
    v = torch.stack(ys, 1).unflatten(2, (G, D // G))
    v = v - v.mean(-1, keepdim=True)
    v = (v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)).flatten(2) * p["gn"] + p["gb"]
    return (v * z * torch.sigmoid(z)) @ p["wout"]


def layer_prompt(p, h):
    proj = h @ p["win"]
    x, gate, i, z = proj.split([D] * 4, -1)         # views of the projection's rows
    xc, conv = m3.mamba3_conv_fwd(x, p["conv"], p["cbias"])
    y, state = m3.mamba3_gated_scan_fwd(xc, gate, p["decay"], i=i)
    n = m3.mamba3_groupnorm_fwd(y, p["gn"], p["gb"], groups=G, z=z, act="gate", eps=EPS)
    return n @ p["wout"], conv, state, (x, gate, i, z, xc, y, n)


def layer_token(p, h, conv, state, slots):
    x, gate, i, z = (h @ p["win"]).split([D] * 4, -1)
    xc = m3.mamba3_conv_step(x, p["conv"], p["cbias"], conv=conv, slots=slots)
    y = m3.mamba3_gated_step(xc, gate, p["decay"], h=state, i=i, slots=slots)
    return m3.mamba3_groupnorm_fwd(y, p["gn"], p["gb"], groups=G, z=z, act="gate", eps=EPS) @ p["wout"]


def near(got, want, what, limit=2e-4):
    got, want = got.cpu().double(), want.detach().cpu().double()
    assert got.shape == want.shape and float((got - want).norm()) <= limit * float(want.norm()) + 1e-12, what


def test_layer_prompt_then_tokens():
    """A prompt, then single tokens over slots, equal the whole; between the two the states go through a cache:
    the tokens after it are those of the states that the cache's reference reads back."""
    g = gen(1)
    b, L, n = 3, 50, 37
    p, h = layer_weights(g), rand(g, b, L, M)
    want = layer_plain({k: v.double() for k, v in p.items()}, h.double())
    q, hd = dev(p), up(h)
    out, conv, state, _ = layer_prompt(q, hd[:, :n].contiguous())
    near(out, want[:, :n], "prompt")
    slots = torch.tensor([4, 0, 6], dtype=torch.int32, device=device())
    for kind in (None, "int8", "int4", "e4m3"):
        cpool, hpool = torch.zeros(7, W - 1, D, device=device()), torch.zeros(7, D, device=device())
        cpool[slots.long()], hpool[slots.long()] = conv, state
        if kind:
            to = torch.tensor([2, 1, 5], dtype=torch.int32, device=device())
            kept = [m3.mamba3_state_store(t, kind=kind, block=32, slots=slots) for t in (cpool, hpool)]
            for (qq, s), t in zip(kept, (cpool, hpool)):
                t.zero_()
                m3.mamba3_state_load(qq, s, h=t, kind=kind, block=32, slots=to)
                src = (conv if t is cpool else state).cpu().flatten(1)
                ref = R.load(*R.store(src, kind, 32), kind, 32, src.shape[1], F32)
                assert torch.equal(t[to.long()].cpu().flatten(1), ref)
        else:
            to = slots
        last = []
        for t in range(n, L):
            last.append(layer_token(q, hd[:, t], cpool, hpool, to))
        if kind is None:
            near(torch.stack(last, 1), want[:, n:], "tokens")
            exact = torch.stack(last, 1)
        else:       # a state of 8 or 4 bits is that near, and its error dies out
            near(torch.stack(last, 1)[:, 0], exact[:, 0], kind, 0.2 if kind == "int4" else 0.05)


def test_layer_gradients():
    g = gen(2)
    b, L = 2, 45
    p, h, dout = layer_weights(g), rand(g, b, L, M), rand(g, b, L, M)
    leaf = {k: v.double().requires_grad_(True) for k, v in dict(p, h=h).items()}
    layer_plain(leaf, leaf["h"]).backward(dout.double())
    q, do = dev(p), up(dout)
    _, _, _, (x, gate, i, z, xc, y, n) = layer_prompt(q, up(h))
    gr = {"wout": n.flatten(0, 1).t() @ do.flatten(0, 1)}
    gn = m3.mamba3_groupnorm_bwd(y, q["gn"], q["gb"], dy=do @ q["wout"].t(), groups=G, z=z, act="gate", eps=EPS)
    gr.update(gn=gn["dweight"], gb=gn["dbias"])
    sc = m3.mamba3_gated_scan_bwd(xc, gate, q["decay"], dy=gn["dx"], i=i)
    gr["decay"] = sc["dweight"]
    cv = m3.mamba3_conv_bwd(x, q["conv"], q["cbias"], dy=sc["dx"])
    gr.update(conv=cv["dweight"], cbias=cv["dbias"])
    dp = torch.cat([cv["dx"], sc["dgate"], sc["di"], gn["dz"]], -1)
    gr.update(win=up(h).flatten(0, 1).t() @ dp.flatten(0, 1), h=dp @ q["win"].t())
    assert set(gr) == set(leaf)
    for k in gr:
        near(gr[k], leaf[k].grad, k)


# ----------------------------------------------------------------------------- calls of every kind, for the tests below
def calls(g, dtype):
    """name -> (inputs, function of them that returns tensors)."""
    out = {}
    for form in ("decay", "forget"):
        for tag, (b, L, cu) in dict(padded=(2, 400, None), packed=(1, 700, [0, 7, 7, 450, 690])).items():
            S = len(cu) - 1 if cu else b
            v = {k: rand(g, b, L, 72, dtype=dtype) for k in ("x", "gate", "i", "z", "dy")}
            v.update(w=rand(g, 72) - 4 if form == "decay" else torch.rand(72, generator=g), h=rand(g, S, 72), dh=rand(g, S, 72))
            if cu:
                v["cu"] = torch.tensor(cu, dtype=torch.int32)
            kw = lambda v, form=form: dict(form=form, i=v["i"], z=v["z"], h_in=v["h"], cu_seqlens=v.get("cu"))   # noqa: E731

            def fwd(v, kw=kw):
                y, h = m3.mamba3_gated_scan_fwd(v["x"], v["gate"], v["w"], y=torch.zeros_like(v["x"]), **kw(v))
                return y, h

            def bwd(v, kw=kw, end=cu[-1] if cu else None):
                r = m3.mamba3_gated_scan_bwd(v["x"], v["gate"], v["w"], dy=v["dy"], dh_out=v["dh"], **kw(v))
                return [t[:, :end] if t.dim() == 3 else t for t in r.values()]

            out[f"scan {form} {tag}"], out[f"scan_bwd {form} {tag}"] = (v, fwd), (v, bwd)
    v = {k: rand(g, 1, 1100, 4096, dtype=dtype) for k in ("x", "gate", "i")}
    v.update(w=rand(g, 4096) - 4, h=rand(g, 1, 4096))
    out["scan one pass"] = (v, lambda v: m3.mamba3_gated_scan_fwd(v["x"], v["gate"], v["w"], i=v["i"], h_in=v["h"]))
    for size in (32, 300, 1500):
        v = {k: rand(g, 37, 2 * size, dtype=dtype) for k in ("x", "z", "dy")}
        v.update(w=rand(g, 2 * size), b=rand(g, 2 * size))
        out[f"norm {size}"] = (v, lambda v: [m3.mamba3_groupnorm_fwd(v["x"], v["w"], v["b"], groups=2, z=v["z"], act="gate")])
        out[f"norm_bwd {size}"] = (v, lambda v: m3.mamba3_groupnorm_bwd(v["x"], v["w"], v["b"], dy=v["dy"], groups=2, z=v["z"],
                                                                      act="pregate").values())
    v = dict(x=rand(g, 5, 72, dtype=dtype), gate=rand(g, 5, 72, dtype=dtype), w=rand(g, 72), h=rand(g, 9, 72),
             slots=torch.tensor([3, -1, 8, 0, 9], dtype=torch.int32))

    def step(v):
        h, y = v["h"].clone(), torch.zeros_like(v["x"])
        return m3.mamba3_gated_step(v["x"], v["gate"], v["w"], h=h, slots=v["slots"], y=y), h

    out["step"] = (v, step)
    v = dict(h=rand(g, 9, 5, 60, dtype=dtype), slots=torch.tensor([3, 1, 8, 0, 9], dtype=torch.int32), to=torch.tensor([1, 2, 3, 4, 5], dtype=torch.int32))

    def cache(v):
        res = []
        for kind in ("e4m3", "int8", "int4"):
            q, s = m3.mamba3_state_store(v["h"], kind=kind, block=32)
            back = m3.mamba3_state_load(q, s, h=torch.zeros_like(v["h"]), kind=kind, block=32, slots=v["to"], entries=v["slots"])
            res += [q.view(torch.uint8), s, back]
        return res

    out["cache"] = (v, cache)
    return out


NAMES = [f"{k} {f} {t}" for k in ("scan", "scan_bwd") for f in ("decay", "forget") for t in ("padded", "packed")] + \
    [f"{k} {s}" for k in ("norm", "norm_bwd") for s in (32, 300, 1500)] + ["step", "cache", "scan one pass"]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("name", NAMES)
def test_captured_and_replayed(name, dtype):
    """A captured call replayed on new inputs, with eager work between the replays, equals the eager call bit for
    bit; two graphs of one call are replayed in turn, and at once on two streams."""
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
        for t in v.values():       # other inputs: the channels of the first ones rolled
            if t.is_floating_point():
                t.copy_(t.roll(1, -1))
        want = [t.clone() for t in f(v)]
        for gr, outs in graphs:
            gr.replay()
            torch.cuda.synchronize()
            for a, b in zip(outs, want):
                assert torch.equal(a, b), (name, k)
            for t in outs:
                t.zero_()
        torch.cuda.synchronize()
        for gr, s in zip(graphs, (torch.cuda.Stream(), torch.cuda.Stream())):
            with torch.cuda.stream(s):
                gr[0].replay()
        torch.cuda.synchronize()
        for _, outs in graphs:
            assert all(torch.equal(a, b) for a, b in zip(outs, want)), (name, k)


@pytest.mark.parametrize("name", NAMES)
def test_on_other_streams(name):
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
    x, gate, w = up(rand(g, 1, 900, 64)), up(rand(g, 1, 900, 64)), up(rand(g, 64))
    s = torch.cuda.Stream()

    def all_(**k):
        y, h = m3.mamba3_gated_scan_fwd(x, gate, w, **k)
        r = [y, h, *m3.mamba3_gated_scan_bwd(x, gate, w, dy=x, **k).values()]
        hs = h.clone()
        r += [m3.mamba3_gated_step(x[:, 0].contiguous(), gate[:, 0].contiguous(), w, h=hs, **k), hs]
        r += [m3.mamba3_groupnorm_fwd(x, w, groups=4, **k), *m3.mamba3_groupnorm_bwd(x, w, dy=x, groups=4, **k).values()]
        q, sc = m3.mamba3_state_store(x[0], **k)
        return r + [q, sc, m3.mamba3_state_load(q, sc, h=torch.zeros_like(x[0]), **k)]

    want = all_()
    torch.cuda.synchronize()
    for which in (s, s.cuda_stream):
        with torch.cuda.stream(s):      # (the test's own clones and zeros lie on it too)
            got = all_(stream=which)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_binding_refusals_on_the_device():
    d = device()
    x, w = torch.zeros(2, 6, 8, device=d), torch.zeros(8, device=d)
    st = torch.zeros(4, 8, device=d)
    i32 = torch.zeros(4, dtype=torch.int32, device=d)
    for bad, err in ((lambda: m3.mamba3_gated_scan_fwd(x, x[:, :5], w), ValueError), (lambda: m3.mamba3_gated_scan_fwd(x, x.bfloat16(), w), TypeError),
                     (lambda: m3.mamba3_gated_scan_fwd(x, x, w.bfloat16()), TypeError), (lambda: m3.mamba3_gated_scan_fwd(x, x, w, form="gru"), ValueError),
                     (lambda: m3.mamba3_gated_scan_fwd(x, x), m3.Mamba3Error), (lambda: m3.mamba3_gated_scan_fwd(x, x, w, rate=-1.0), m3.Mamba3Error),
                     (lambda: m3.mamba3_gated_scan_fwd(x, x, w, y=x), m3.Mamba3Error), (lambda: m3.mamba3_gated_scan_fwd(x, x, w, h_in=st), ValueError),
                     (lambda: m3.mamba3_gated_scan_fwd(x, x, w, cu_seqlens=i32), ValueError), (lambda: m3.mamba3_gated_scan_fwd(x.half(), x.half(), w), TypeError),
                     (lambda: m3.mamba3_gated_scan_bwd(x, x, w, dy=x[:1]), ValueError),
                     (lambda: m3.mamba3_gated_scan_bwd(x, x, w, dy=x, workspace=torch.zeros(256, dtype=torch.uint8, device=d)), m3.Mamba3Error),
                     (lambda: m3.mamba3_gated_step(x[0], x[0], w, h=st), ValueError), (lambda: m3.mamba3_gated_step(x[0], x[0], w, h=st, slots=i32), ValueError),
                     (lambda: m3.mamba3_groupnorm_fwd(x, w, groups=3), m3.Mamba3Error), (lambda: m3.mamba3_groupnorm_fwd(x, w, groups=2, act="gate"), m3.Mamba3Error),
                     (lambda: m3.mamba3_groupnorm_fwd(x, w, groups=2, z=x), m3.Mamba3Error), (lambda: m3.mamba3_groupnorm_fwd(x, st[0, :4], groups=2), ValueError),
                     (lambda: m3.mamba3_groupnorm_fwd(torch.zeros(2, 8200, device=d), groups=1), m3.Mamba3Error),
                     (lambda: m3.mamba3_state_store(st, block=16), ValueError), (lambda: m3.mamba3_state_store(st, kind="fp4"), ValueError),
                     (lambda: m3.mamba3_state_store(st, entries=i32), ValueError), (lambda: m3.mamba3_state_store(st, slots=i32.long()), TypeError),
                     (lambda: m3.mamba3_state_store(st.half()), TypeError), (lambda: m3.mamba3_state_store(st.t()), ValueError),
                     (lambda: m3.mamba3_state_store(st, slots=i32, entries=i32[:3], q=torch.zeros(4, 8, dtype=torch.int8, device=d),
                                                    scale=torch.zeros(4, 1, device=d)), ValueError),
                     (lambda: m3.mamba3_state_load(torch.zeros(3, 8, dtype=torch.int8, device=d), torch.zeros(3, 1, device=d), h=st), ValueError),
                     (lambda: m3.mamba3_state_load(torch.zeros(4, 8, dtype=torch.uint8, device=d), torch.zeros(4, 1, device=d), h=st), TypeError),
                     (lambda: m3.mamba3_state_load(torch.zeros(4, 7, dtype=torch.int8, device=d), torch.zeros(4, 1, device=d), h=st), ValueError),
                     (lambda: m3.mamba3_state_load(torch.zeros(4, 8, dtype=torch.int8, device=d), torch.zeros(4, 2, device=d), h=st), ValueError)):
        with pytest.raises(err):
            bad()


# ----------------------------------------------------------------------------- past 32 bits
T, C, TAIL = (1 << 20) + 3, 4096, 400


def test_arrays_past_the_32_bits():
    """Token arrays of more than 2^32 elements: the first and last tokens of the gated scan, the group norm and their
    gradients. (Least decay 0: a state forgets what lies 200 tokens back, gates of 0.5 and below.)"""
    note(f"{T} tokens of {C} channels")
    g = torch.Generator(device=device()).manual_seed(8)
    x = torch.empty((1, T, C), dtype=BF16, device=device())
    for k in range(0, T, 1 << 18):
        x[:, k:k + (1 << 18)] = torch.randn(x[:, k:k + (1 << 18)].shape, generator=g, device=device(), dtype=BF16)
    gate = -x.abs()
    ends = ((0, 0, TAIL - 200), (T - TAIL, 200, TAIL))       # a slice's first token, and its tokens that are compared
    cut = lambda t, a: t[:, a:a + TAIL].cpu()   # noqa: E731

    def compare(got, ref, names, a, lo, hi):
        for k in names:
            assert R.off(cut(got[k], a)[:, lo:hi], tuple(t[:, lo:hi] for t in ref[k])) <= 1, (k, a)

    y, h = m3.mamba3_gated_scan_fwd(x, gate, form="forget", i=x, z=x)
    refs = {a: R.scan(cut(x, a), cut(gate, a), None, "forget", 8.0, cut(x, a), cut(x, a), None, None, cut(x, a)) for a, _, _ in ends}
    for a, lo, hi in ends:
        compare(dict(y=y), refs[a], ("y",), a, lo, hi)
    assert R.off(h, refs[T - TAIL]["h_out"]) <= 1
    del y
    gr = m3.mamba3_gated_scan_bwd(x, gate, form="forget", i=x, z=x, dy=x)
    # (a gradient comes from behind: the first slice's own end is cut, the last one's is the sequence's)
    for a, lo, hi in ends:
        compare(gr, refs[a], ("dx", "dgate", "di", "dz"), a, lo, hi)
    del gr
    w = up(rand(gen(1), C))
    y = m3.mamba3_groupnorm_fwd(x, w, groups=32, z=x, act="gate")
    gr = m3.mamba3_groupnorm_bwd(x, w, groups=32, z=x, act="gate", dy=x)
    for a, _, _ in ends:
        s = cut(x, a)[0]
        ref = R.groupnorm(s, w.cpu(), None, 32, s, "gate", True, 1e-5, s)
        for k, t in (("y", y), ("dx", gr["dx"]), ("dz", gr["dz"])):
            assert R.off(cut(t, a)[0], ref[k]) <= 1, (k, a)


def test_caches_past_the_32_bits():
    """Slots and entries more than 2^32 bytes into the pool and the cache."""
    values, n = 1 << 20, 5000
    pool = torch.empty((1300, values), device=device())
    note(f"pool of {pool.numel() * 4 >> 20} MiB")
    slots = torch.tensor([1299, 3, 1100, 1300], dtype=torch.int32, device=device())
    entries = torch.tensor([4999, 7, 4100, 1], dtype=torch.int32, device=device())
    h = rand(gen(4), 3, values)
    pool[slots[:3].long()] = up(h)
    for kind in ("int8", "int4"):
        q = torch.empty((n, values // (2 if kind == "int4" else 1)), dtype=torch.int8 if kind == "int8" else torch.uint8, device=device())
        s = torch.empty((n, values // 256), device=device())
        m3.mamba3_state_store(pool, kind=kind, block=256, slots=slots, entries=entries, q=q, scale=s)
        want, scale = R.store(h, kind, 256)
        assert torch.equal(q[entries[:3].long()].cpu(), want) and torch.equal(s[entries[:3].long()].cpu(), scale)
        to = torch.tensor([1200, 1250, 0, 2], dtype=torch.int32, device=device())
        m3.mamba3_state_load(q, s, h=pool, kind=kind, block=256, slots=to[:3], entries=entries[:3])
        assert torch.equal(pool[to[:3].long()].cpu(), R.load(want, scale, kind, 256, values, F32))


def test_step_pool_past_the_32_bits():
    pool = torch.zeros((300001, 4096), device=device())
    slots = torch.tensor([300000, 5, 299999, 300001], dtype=torch.int32, device=device())
    g = gen(7)
    x, gate, w, start = rand(g, 4, 4096, dtype=BF16), rand(g, 4, 4096, dtype=BF16), rand(g, 4096), rand(g, 4, 4096)
    pool[slots[:3].long()] = up(start)[:3]
    own = up(start)
    y = m3.mamba3_gated_step(up(x), up(gate), up(w), h=pool, slots=slots)
    want = m3.mamba3_gated_step(up(x), up(gate), up(w), h=own)
    assert torch.equal(y[:3], want[:3]) and torch.equal(pool[slots[:3].long()], own[:3])
