"""The gated layer's 64-bit forms on the CPU: their gradients against differences and automatic
differentiation of plain formulas, and that their bounds hold planted mistakes out."""
import pytest
import torch

from tests import gated_ref as R


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rand(g, *shape, std=1.0):
    return torch.randn(shape, generator=g) * std


def scan_case(form, cu=None, b=2, L=23, D=5, seed=0):
    g = gen(seed)
    S = len(cu) - 1 if cu else b
    w = rand(g, D) - 3 if form == "decay" else torch.rand(D, generator=g) * 0.8
    return dict(x=rand(g, b, L, D), gate=rand(g, b, L, D), weight=w, form=form, rate=8.0, i=rand(g, b, L, D),
                z=rand(g, b, L, D), h_in=rand(g, S, D), cu=cu), dict(dy=rand(g, b, L, D), dh_out=rand(g, S, D))


def plain(c):
    """y and the last states from the formulas, differentiable, in 64 bits."""
    w, s = c["weight"], torch.sigmoid(c["gate"])
    if c["form"] == "decay":
        a = torch.exp(-c["rate"] * torch.nn.functional.softplus(w) * s)
        u = torch.sqrt(1 - a * a)
    else:
        a = w + (1 - w) * s
        u = 1 - a
    b = (u * torch.sigmoid(c["i"]) * c["x"]).reshape(-1, w.numel())
    a, z = a.reshape(-1, w.numel()), c["z"].reshape(-1, w.numel())
    ys, ends = [], []
    for q, (t0, t1) in enumerate(R.spans(c["x"].shape[:2], c["cu"])):
        h = c["h_in"][q]
        for t in range(t0, t1):
            h = a[t] * h + b[t]
            ys.append(h * z[t] * torch.sigmoid(z[t]))
        ends.append(h)
    return torch.stack(ys), torch.stack(ends)


@pytest.mark.parametrize("form", ["decay", "forget"])
@pytest.mark.parametrize("cu", [None, [0, 0, 7, 8, 46]])
def test_scan_gradients(form, cu):
    c, back = scan_case(form, cu, *((1, 46) if cu else (2, 23)))
    ref = R.scan(**c, **back)
    d = {k: v.double().requires_grad_(True) if torch.is_tensor(v) else v for k, v in c.items()}

    def loss():
        y, e = plain(d)
        return (y * back["dy"].double().reshape(y.shape)).sum() + (e * back["dh_out"].double()).sum()

    y, e = plain(d)
    assert torch.allclose(y.reshape(c["x"].shape), ref["y"][0], rtol=1e-12, atol=1e-14)
    assert torch.allclose(e, ref["h_out"][0], rtol=1e-12, atol=1e-14)
    loss().backward()
    for k, name in (("x", "dx"), ("gate", "dgate"), ("i", "di"), ("z", "dz"), ("weight", "dweight"), ("h_in", "dh_in")):
        assert torch.allclose(d[k].grad, ref[name][0], rtol=1e-9, atol=1e-11), name
        # and differences, in one direction
        v = torch.randn(d[k].shape, generator=gen(9)).double()
        step = 1e-6
        with torch.no_grad():
            d[k] += step * v
            up = loss()
            d[k] -= 2 * step * v
            down = loss()
            d[k] += step * v
        want = float((ref[name][0] * v).sum())
        assert abs(float(up - down) / (2 * step) - want) <= 1e-6 * (1 + abs(want)), name


@pytest.mark.parametrize("act", ["none", "silu", "gate", "pregate"])
@pytest.mark.parametrize("center", [True, False])
def test_groupnorm_gradients(act, center):
    g = gen(4)
    x, w, b, dy = rand(g, 7, 30), rand(g, 30), rand(g, 30), rand(g, 7, 30)
    z = rand(g, 7, 30) if "gate" in act else None
    ref = R.groupnorm(x, w, b, 3, z, act, center, 1e-3, dy)
    p = {k: v.double().requires_grad_(True) for k, v in dict(x=x, w=w, b=b, z=z).items() if v is not None}

    def loss():
        t = p["x"] * torch.nn.functional.silu(p["z"]) if act == "pregate" else p["x"]
        t = t.view(7, 3, 10)
        if center:
            t = t - t.mean(-1, keepdim=True)
        v = (t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-3)).reshape(7, 30) * p["w"] + p["b"]
        if act == "silu":
            v = torch.nn.functional.silu(v)
        if act == "gate":
            v = v * torch.nn.functional.silu(p["z"])
        return v

    assert torch.allclose(loss(), ref["y"][0], rtol=1e-12, atol=1e-13)
    (loss() * dy.double()).sum().backward()
    for k, name in (("x", "dx"), ("w", "dweight"), ("b", "dbias"), ("z", "dz")):
        if k not in p:
            continue
        assert torch.allclose(p[k].grad, ref[name][0], rtol=1e-9, atol=1e-11), name
        v = torch.randn(p[k].shape, generator=gen(9)).double()
        step = 1e-6
        with torch.no_grad():
            p[k] += step * v
            up = (loss() * dy.double()).sum()
            p[k] -= 2 * step * v
            down = (loss() * dy.double()).sum()
            p[k] += step * v
        want = float((ref[name][0] * v).sum())
        assert abs(float(up - down) / (2 * step) - want) <= 1e-6 * (1 + abs(want)), name


@pytest.mark.parametrize("form", ["decay", "forget"])
def test_bounds_hold_mistakes_out(form):
    """A state or gradient rounded to bf16 once, a decay that missed a token: outside the bounds of fp32
    outputs. An fp32 evaluation of the formulas is inside."""
    c, back = scan_case(form, None, 1, 96, 6, seed=3)
    if form == "forget":
        c["gate"] = c["gate"] + 3
    ref = R.scan(**c, **back)
    rough = lambda v: v.float().bfloat16().double()   # noqa: E731
    # near the end that the outputs lie at: decays wash a mistake out on the way
    for which, place, names in (("h", 90, ("y", "h_out", "dgate")), ("g", 5, ("dx", "dgate", "dh_in"))):
        bad = R.scan(**c, **back, spoil=lambda what, t, v: rough(v) if what == which and t == place else v)   # noqa: B023
        for k in names:
            assert R.off(bad[k][0].float(), ref[k]) > 2, (which, k)
    y32, e32 = plain({k: v.float() if torch.is_tensor(v) else v for k, v in c.items()})
    if form == "forget":        # (1 - a^2 by subtraction is not what the bound stands for)
        assert R.off(y32.reshape(c["x"].shape), ref["y"]) <= 1 and R.off(e32, ref["h_out"]) <= 1


def test_cache_reference():
    """Every byte of the kinds reads back as what it stands for, and values that are scaled bytes already come back
    whole."""
    g = gen(2)
    for kind, low, high in (("int8", -127, 127), ("int4", -7, 7)):
        v = torch.randint(low, high + 1, (3, 101), generator=g).float()
        v[:, ::32] = high
        q, s = R.store(v * 0.25, kind, 32)
        assert torch.equal(s, torch.full((3, 4), 0.25))
        assert torch.equal(R.load(q, s, kind, 32, 101, torch.float32), v * 0.25)
    v = torch.randn(2, 70, generator=g)
    q, s = R.store(v, "e4m3", 64)
    back = R.load(q, s, "e4m3", 64, 70, torch.float32)
    least = s.repeat_interleave(64, 1)[:, :70] * 2.0 ** -10       # half the least subnormal
    assert bool(((back - v).abs() <= v.abs() * 2.0 ** -4 * 1.001 + least).all())
    v[0, 3] = float("inf")
    q, s = R.store(v, "int8", 64)
    back = R.load(q, s, "int8", 64, 70, torch.float32)
    assert bool(back[0, :64].isnan().all()) and bool(back[0, 64:].isfinite().all()) and bool(back[1].isfinite().all())
