"""Plain 64-bit forms of the layer operators for the tests: one sequence at a time, one token at a time,
on the CPU. With ``mag`` a function computes the same sums over the terms' absolute values, which is
what the roundings of a 32-bit computation are relative to."""
import torch

U32 = 2.0 ** -24        # half a step of fp32, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def within(got, ref, mag, count, what):
    """got is ref rounded once to its type, computed in fp32 from terms of magnitude `mag` with `count`
    roundings on the way. (Subnormal and zero results: the smallest fp32 normal is let pass.)"""
    got, ref = got.detach().cpu().double(), ref.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    both = torch.isnan(got) & torch.isnan(ref) | (got == ref)
    return got, ref, both


def check(got, ref, mag, count, what):
    half = half_step(got.dtype) if got.dtype.is_floating_point else 0.0
    g, r, same = within(got, ref, mag, count, what)
    bound = half * r.abs() * (1 + 4 * count * U32) + count * U32 * mag.double().abs() * (1 + half) + 1e-37
    bad = ~same & ~((g - r).abs() <= bound)
    if bad.any():
        i = int(((g - r).abs() / bound).nan_to_num(1e30).masked_fill(same, 0).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, worst at {i}: got "
                             f"{float(g.flatten()[i])!r}, expected {float(r.flatten()[i])!r}, allowed "
                             f"{float(bound.flatten()[i])!r}")


def silu(v):
    return v / (1 + torch.exp(-v))


def dsilu(v):
    s = 1 / (1 + torch.exp(-v))
    return s + v * s * (1 - s)


def dsilu_terms(v):
    """The size of the terms that dsilu adds: near v = -1.278 they cancel, and a computed dsilu is off by
    roundings of s and |v| s (1 - s), not of their difference."""
    s = 1 / (1 + torch.exp(-v))
    return s + v.abs() * s * (1 - s)


def spans(lead, cu):
    """[(first, last)] of the sequences in token rows laid end to end."""
    b, L = lead
    at = [int(v) for v in cu] if cu is not None else [i * L for i in range(b + 1)]
    return list(zip(at[:-1], at[1:]))


def stack(rows, *shape):
    return torch.stack(rows) if rows else torch.zeros(0, *shape).double()


def conv(x, w, bias, act, conv_in, cu, dy=None, dconv_out=None, mag=False):
    """y and conv_out, and with dy the gradients."""
    f = (lambda t: t.double().abs()) if mag else (lambda t: t.double())
    lead, D, W = x.shape[:2], x.shape[2], w.shape[1]
    flat, wd, bd = f(x).reshape(-1, D), f(w), f(bias) if bias is not None else torch.zeros(D).double()
    tx, tw, tb = x.double().reshape(-1, D), w.double(), bias.double() if bias is not None else torch.zeros(D).double()
    y = torch.zeros_like(flat)
    outs, dins = [], []
    dx, dw, db = torch.zeros_like(flat), torch.zeros(D, W).double(), torch.zeros(D).double()
    for i, (a, b) in enumerate(spans(lead, cu)):
        h = torch.cat([f(conv_in[i]) if conv_in is not None else torch.zeros(W - 1, D).double(), flat[a:b]])
        th = torch.cat([conv_in[i].double() if conv_in is not None else torch.zeros(W - 1, D).double(), tx[a:b]])
        dh = torch.zeros_like(h)
        for t in range(b - a):
            p = bd + sum(wd[:, j] * h[t + j] for j in range(W))
            tp = tb + sum(tw[:, j] * th[t + j] for j in range(W))   # the true value that the activation sees
            y[a + t] = (1.1 * p if mag else silu(p)) if act else p   # |SiLU'| <= 1.1, |SiLU(v)| <= |v|
            if dy is not None:
                e = f(dy.reshape(-1, D)[a + t])
                if act:     # SiLU'' is at most 0.5: an error of p moves e by as much
                    e = e * (dsilu_terms(tp) + 0.5 * p) if mag else e * dsilu(tp)
                db += e
                for j in range(W):
                    dw[:, j] += e * h[t + j]
                    dh[t + j] += e * wd[:, j]
        outs.append(th[b - a:])
        if dconv_out is not None:
            dh[b - a:] += f(dconv_out[i])
        dx[a:b] = dh[W - 1:]
        dins.append(dh[:W - 1])
    r = dict(y=y.view(x.shape), conv_out=stack(outs, W - 1, D))
    if dy is not None:
        r.update(dx=dx.view(x.shape), dweight=dw, dbias=db, dconv_in=stack(dins, W - 1, D))
    return r


def scan(x, dt, A, B, C, D, z, bias, softplus, h_in, cu, dy=None, dh_out=None, mag=False):
    """y and h_out, and with dy the gradients."""
    f = (lambda t: t.double().abs()) if mag else (lambda t: t.double())
    lead, dim, (G, N) = x.shape[:2], x.shape[2], B.shape[2:]
    fl = lambda t: t.double().reshape(-1, *t.shape[2:])   # noqa: E731
    of = torch.arange(dim) // (dim // G)
    fx, fB, fC, Ad = f(fl(x)), f(fl(B)), f(fl(C)), A.double()
    raw = fl(dt) + (bias.double() if bias is not None else 0)
    s = torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw
    gate = 1 / (1 + torch.exp(-raw)) if softplus else torch.ones_like(raw)
    sf = f(s)
    zd = fl(z) if z is not None else None
    Dd = f(D) if D is not None else torch.zeros(dim).double()
    Aw = f(A)
    nd = fl(dy) if dy is not None else None
    y = torch.zeros_like(fx)
    hs = []
    out = {k: torch.zeros_like(v) for k, v in dict(dx=fx, ddt=fx, dz=fx, dB=fB, dC=fC, dA=Ad, dD=Dd,
                                                     ddt_bias=Dd).items()}
    dins = []
    for i, (a, b) in enumerate(spans(lead, cu)):
        h = f(h_in[i]) if h_in is not None else torch.zeros(dim, N).double()
        kept, ys = [], []
        for t in range(a, b):
            kept.append(h)
            h = torch.exp(s[t][:, None] * Ad) * h + (sf[t] * fx[t])[:, None] * fB[t][of]
            yt = (h * fC[t][of]).sum(-1) + Dd * fx[t]
            ys.append((h, yt))
            y[t] = yt * f(silu(zd[t])) if zd is not None else yt
        hs.append(h)
        if dy is None:
            continue
        g = f(dh_out[i]) if dh_out is not None else torch.zeros(dim, N).double()
        for t in range(b - 1, a - 1, -1):
            ht, yt = ys[t - a]
            r = f(nd[t] * silu(zd[t])) if zd is not None else f(nd[t])
            g = g + r[:, None] * fC[t][of]
            if zd is not None:
                out["dz"][t] = (nd[t].abs() * dsilu_terms(zd[t]) if mag else nd[t] * dsilu(zd[t])) * yt
            out["dC"][t] = (r[:, None] * ht).view(G, -1, N).sum(1)
            out["dB"][t] = (g * (sf[t] * fx[t])[:, None]).view(G, -1, N).sum(1)
            gb = (g * fB[t][of]).sum(-1)
            q = g * torch.exp(s[t][:, None] * Ad)
            w = q * kept[t - a]
            out["dA"] += w * sf[t][:, None]
            ds = (gb * fx[t] + (w * Aw).sum(-1)) * gate[t]
            out["ddt"][t] = ds
            out["ddt_bias"] += ds
            out["dx"][t] = gb * sf[t] + Dd * r
            out["dD"] += r * fx[t]
            g = q
        dins.append(g)
    r = dict(y=y.view(x.shape), h_out=stack(hs, dim, N))
    if dy is not None:
        for k in ("dx", "ddt", "dz"):
            out[k] = out[k].view(x.shape)
        out["dB"], out["dC"] = out["dB"].view(B.shape), out["dC"].view(B.shape)
        r.update(out, dh_in=stack(dins, dim, N))
    return r


def norm(x, res, w, eps):
    """s, v and the sum of squares' mean."""
    s = x.double() + (res.double() if res is not None else 0)
    v = s / torch.sqrt((s ** 2).mean(-1, keepdim=True) + eps)
    return s, v * w.double() if w is not None else v


def norm_bwd(s, w, dy, dres, eps, mag=False):
    s, dy = s.double(), dy.double()
    wd = dy * (w.double() if w is not None else 1)
    r = 1 / torch.sqrt((s ** 2).mean(-1, keepdim=True) + eps)
    if mag:
        s, wd, dy = s.abs(), wd.abs(), dy.abs()
    sh = s * r
    first, second = r * wd, r * sh * (wd * sh).mean(-1, keepdim=True)
    ds = first + second if mag else first - second
    if dres is not None:
        ds = ds + (dres.double().abs() if mag else dres.double())
    return ds, (dy * sh).reshape(-1, s.shape[-1]).sum(0)
