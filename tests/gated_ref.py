"""The gated layer's operators in 64 bits on the CPU, token by token and row by row, each result with a
bound on what an fp32 computation of it may be off by: name -> (value, error in units of 2^-24).

The bounds are counted along the computations: a product, sum, division or fused multiply-add is off by one
rounding of its result, a hardware exp2, log2, reciprocal or square root by two; an exponent's own error
counts by its size, and errors of a state run through its recurrence, whose decays shrink them."""
import torch

from tests.layer_bounds import off   # noqa: F401  (the tests' measure)
from tests.layer_ref import spans


def sigmoid(v):
    """sigmoid(v), 1 - sigmoid(v) and their relative errors: the exponent's product and constant (2 |v|), exp2,
    the sum, the reciprocal and a product. One below 2^-126 may count as zero."""
    s, n = 1 / (1 + torch.exp(-v)), 1 / (1 + torch.exp(v))
    k, all_ = 2 * v.abs() + 6, torch.full_like(v, 2.0 ** 24)
    return s, n, torch.where(s < 2.0 ** -125, all_, k), torch.where(n < 2.0 ** -125, all_, k)


def silu(z):
    """SiLU, its relative error, its derivative and the error of that."""
    s, n, k, _ = sigmoid(z)
    d, terms = s * (1 + z * n), s * (1 + z.abs() * n)
    # 1 - s by a subtraction: off by s's error and a rounding, both relative to one; then two operations and a product
    ed = s * (1 + z.abs() * n) * k + s * z.abs() * (s * k + 2) + 3 * terms
    return z * s, k + 1, d, ed


def gates(g, w, form, rate):
    """a, u, 1 / u (0 for u = 0), log a (decay form), sigmoid and its complement, and the relative errors of a, u, the
    sigmoid, its complement and log a."""
    s, n, ks, kn = sigmoid(g)
    if form == "decay":
        soft = torch.logaddexp(w, torch.zeros_like(w))
        la = -rate * soft * s
        kl = ks + 12                        # softplus by exp, log, a reciprocal and their corrections, times rate, times s
        a = torch.exp(la)
        ka = la.abs() * (kl + 3) + 2
        sq = -torch.expm1(2 * la)
        # the series: la's error and its own roundings; the difference: twice a's, over 1 - a^2
        kw = torch.where(la > -0.126, kl + 10, 2 * ka * a * a / sq.clamp(min=1e-300) + 3)
        u = torch.sqrt(sq)
        # a subnormal 1 - a^2 may count as zero
        ku = torch.where(sq < 2.0 ** -125, torch.full_like(sq, 2.0 ** 24), kw / 2 + 3)
    else:
        l = w if w is not None else torch.zeros(g.shape[-1]).double()
        u = (1 - l) * n
        a = l + (1 - l) * s
        la, kl = None, None
        ka, ku = ks.minimum(2 * g.abs() + 6) + 3, kn + 2       # (a sum with l, or zero itself)
    inv = torch.where(u > 0, 1 / u.clamp(min=1e-300), torch.zeros_like(u))
    return a, u, inv, la, s, n, ka, ku, ks, kn, kl


def scan(x, gate, weight, form, rate, i, z, h_in, cu, dy=None, dh_out=None, spoil=None):
    """`spoil(which, token, value)` may change the state that enters a token ("h") or the gradient that leaves
    it ("g"): a planted mistake."""
    spoil = spoil or (lambda what, t, v: v)
    lead, D = x.shape[:2], x.shape[2]
    fl = lambda t: t.double().reshape(-1, D)   # noqa: E731
    T = lead[0] * lead[1]
    w = weight.double() if weight is not None else None
    a, u, inv, la, s, n, ka, ku, ks, kc, kl = gates(fl(gate), w, form, rate)
    xd = fl(x)
    si, ni, ki, kj = sigmoid(fl(i)) if i is not None else (torch.ones_like(xd), None, torch.zeros_like(xd), None)
    v, kv = si * xd, ki + 1
    b, kb = u * v, ku + kv + 1
    zd = fl(z) if z is not None else None
    sz, kz, dsz, edsz = silu(zd) if z is not None else (torch.ones_like(xd), torch.zeros_like(xd), None, None)
    names = ["y"] + (["dx", "dgate", "di", "dz"] if dy is not None else [])
    V = {k: torch.zeros(T, D).double() for k in names}
    E = {k: torch.zeros(T, D).double() for k in names}
    dw, dwe, dwm = (torch.zeros(D).double() for _ in range(3))
    ends, dins = [], []
    zero = torch.zeros(D).double()
    rd = fl(dy) if dy is not None else None
    for q, (t0, t1) in enumerate(spans(lead, cu)):
        h = h_in[q].double() if h_in is not None else zero
        hm, he = h.abs(), zero
        kept = []
        for t in range(t0, t1):
            h = spoil("h", t - t0, h)
            kept.append((h, hm, he))
            # the product of decays and the state of a run are joined to what enters it: three more roundings
            # a token at most
            he = a[t] * he + a[t] * hm * (ka[t] + 4) + b[t].abs() * (kb[t] + 1)
            h, hm = a[t] * h + b[t], a[t] * hm + b[t].abs()
            he = he + hm
            V["y"][t], E["y"][t] = h * sz[t], he * sz[t].abs() + hm * sz[t].abs() * (kz[t] + 1)
        ends.append((h, he))
        kept.append((h, hm, he))
        if dy is None:
            continue
        g = dh_out[q].double() if dh_out is not None else zero
        gm, ge = g.abs(), zero
        for t in range(t1 - 1, t0 - 1, -1):
            hp, hpm, hpe = kept[t - t0]
            hn, hnm, hne = kept[t - t0 + 1]
            g = spoil("g", t - t0, g)
            r, kr = rd[t] * sz[t], kz[t] + 1
            if z is not None:
                V["dz"][t] = rd[t] * hn * dsz[t]
                E["dz"][t] = rd[t].abs() * (hne * dsz[t].abs() + hnm * edsz[t] + 2 * hnm * dsz[t].abs())
            G, Gm = g + r, gm + r.abs()
            Ge = ge + r.abs() * kr + Gm
            dv, dvm = u[t] * G, u[t] * Gm
            dve = u[t] * Ge + dvm * (ku[t] + 1)
            V["dx"][t], E["dx"][t] = dv * si[t], dve * si[t] + dvm * si[t] * (ki[t] + 1)
            if i is not None:
                V["di"][t] = dv * v[t] * ni[t]
                E["di"][t] = (dve + dvm * (kv[t] + kj[t] + 4)) * (v[t] * ni[t]).abs()
            if form == "decay":
                f, kf = (a[t] * la[t]).abs(), ka[t] + kl[t] + 1
                back = v[t] * a[t] * inv[t]
                inner, im = hp - back, hpm + back.abs()
                ie = hpe + back.abs() * (kv[t] + ka[t] + ku[t] + 4) + im
                Q = G * a[t] * la[t] * inner
                V["dgate"][t], mul, kn = Q * n[t], n[t], kc[t] + 1
            else:
                f, kf = n[t], kc[t]
                inner, im = hp - v[t], hpm + v[t].abs()
                ie = hpe + v[t].abs() * kv[t] + im
                Q = G * inner * n[t]
                sl = (1 - w if w is not None else 1) * s[t]
                V["dgate"][t], mul, kn = Q * sl, sl, ks[t] + 3
            Qm = Gm * f * im
            Qe = Ge * f * im + Gm * f * ie + Qm * (kf + 2)
            E["dgate"][t] = (Qe + Qm * kn) * mul
            dw += Q
            # 16 additions a run's share, runs one by one over 16 threads
            dwe += Qe + Qm
            dwm += Qm
            g, gm = a[t] * G, a[t] * Gm
            ge = a[t] * Ge + gm * (ka[t] + 4)
        dins.append((g, ge + gm))
    out = {k: (V[k].view(x.shape), E[k].view(x.shape)) for k in names}
    for k, rows in (("h_out", ends),) + ((("dh_in", dins),) if dy is not None else ()):
        out[k] = tuple(torch.stack([p[j] for p in rows]) if rows else torch.zeros(0, D).double() for j in (0, 1))
    if dy is not None:
        depth = 8 + 8 + T / 32 / 16 + len(ends) / 16 + 18      # a lane, the waves, the rows of a thread, 16 threads
        if form == "decay":
            ratio = torch.sigmoid(w) / torch.logaddexp(w, torch.zeros_like(w))
            out["dweight"] = dw * ratio, (dwe + dwm * (depth + 20)) * ratio
        else:
            out["dweight"] = dw, dwe + dwm * depth
    return out


# ----------------------------------------------------------------------------- group norm
# Additions on the longest path of a group's sum: 8 values of a lane, 6 levels over a wave, 16 waves
DEPTH = 8 + 6 + 16


def groupnorm(x, weight, bias, groups, z, act, center, eps, dy=None):
    dim = x.shape[-1]
    shape = (-1, groups, dim // groups)
    sh = lambda t: t.double().reshape(shape)   # noqa: E731
    one = torch.ones(dim).double()
    w = (weight.double() if weight is not None else one).view(shape[1:])
    b = (bias.double() if bias is not None else 0 * one).view(shape[1:])
    X = sh(x)
    mean = lambda t: t.mean(-1, keepdim=True)   # noqa: E731
    if z is not None:
        Z = sh(z)
        sz, kz, dsz, edsz = silu(Z)
    if act == "pregate":
        t, te = X * sz, (X * sz).abs() * (kz + 1)
    else:
        t, te = X, torch.zeros_like(X)
    m = mean(t) if center else torch.zeros_like(t[..., :1])
    var = mean((t - m) ** 2) + eps
    r = 1 / torch.sqrt(var)
    n = (t - m) * r
    # what is left of the mean's rounding is taken off once more, with the error of a sum of differences; a
    # far mean's own rounding comes in by its square
    far = (DEPTH + 4) * 2.0 ** -24 * mean(t.abs()) * r if center else 0 * r
    nm = mean(n.abs())
    ne = 3 * n.abs() + te * r
    if center:
        ne = ne + (DEPTH + 4) * nm + mean(te) * r
    # 1 / deviation: the sum of squares and what moves them, halved
    rel = (DEPTH + 6) / 2 + 4 + mean(n.abs() * ne) + far ** 2 * 2.0 ** 24
    ne = ne + n.abs() * rel
    v, vm = n * w + b, (n * w).abs() + b.abs()
    ve = ne * w.abs() + (n * w).abs() * 2 + vm
    out = {}
    if act == "silu":
        sv, _, dsv, edsv = silu(v)
        # an error of v comes through with SiLU's slope, at most 1.1
        y, ye = sv, 1.1 * ve + sv.abs() * (2 * v.abs() + 8)
    elif act == "gate":
        y, ye = v * sz, ve * sz.abs() + vm * sz.abs() * (kz + 1)
    else:
        y, ye = v, ve
    out["y"] = y, ye
    if dy is not None:
        d, de = sh(dy), torch.zeros_like(X)
        if act == "silu":
            # SiLU'' is at most 1/2
            d, de = d * dsv, d.abs() * (edsv + 0.5 * ve + dsv.abs())
        elif act == "gate":
            out["dz"] = d * v * dsz, d.abs() * (ve * dsz.abs() + vm * edsz + 2 * vm * dsz.abs())
            d, de = d * sz, (d * sz).abs() * (kz + 1)
        rows = X.shape[0]
        walk = rows / 64 + 64 + 40        # rows of a lane, of 16 threads, the workgroup's waves and the threads
        out["dbias"] = d.sum(0), de.sum(0) + walk * d.abs().sum(0)
        out["dweight"] = (d * n).sum(0), (de * n.abs() + d.abs() * ne).sum(0) + (walk + 1) * (d * n).abs().sum(0)
        dn, dne = d * w, (de + d.abs()) * w.abs()
        s1, s2 = mean(dn) if center else 0 * r, mean(dn * n)
        e1 = (mean(dne) + DEPTH * mean(dn.abs())) if center else 0 * r
        e2 = mean(dne * n.abs() + dn.abs() * ne) + (DEPTH + 2) * mean((dn * n).abs())
        dt = r * (dn - s1 - n * s2)
        mag = dn.abs() + s1.abs() + (n * s2).abs()
        dte = r * (dne + e1 + n.abs() * e2 + ne * s2.abs() + 4 * mag + mag * (rel + 2))
        if act == "pregate":
            out["dz"] = dt * X * dsz, dte * (X * dsz).abs() + r * mag * X.abs() * (edsz + 2 * dsz.abs())
            dt, dte = dt * sz, dte * sz.abs() + r * mag * sz.abs() * (kz + 1)
        out["dx"] = dt, dte
    flat = {"dweight": (dim,), "dbias": (dim,)}
    return {k: tuple(q.reshape(flat.get(k, x.shape)) for q in p) for k, p in out.items()}


# ----------------------------------------------------------------------------- state cache
TOP = {"e4m3": 448.0, "int8": 127.0, "int4": 7.0}


def store(h, kind, block):
    """(q as the cache holds it, scale) of states [n, values]: every rounding as documented."""
    n, m = h.shape
    blocks = -(-m // block)
    v = torch.zeros(n, blocks * block)
    v[:, :m] = h.float()
    v = v.view(n, blocks, block)
    top = v.abs().amax(-1)
    # (a quotient of two fp32 numbers, rounded from 64 bits, is the rounded quotient)
    scale = (top.double() / TOP[kind]).float().clamp(min=2.0 ** -126)
    scale[~torch.isfinite(top)] = float("nan")
    q = (v.double() / scale[..., None].double()).float().reshape(n, -1)[:, :m]
    if kind == "e4m3":
        return q.to(torch.float8_e4m3fn), scale
    q = torch.round(q).clamp(-TOP[kind], TOP[kind]).nan_to_num(-TOP[kind])
    if kind == "int8":
        return q.to(torch.int8), scale
    q = torch.cat([q, torch.zeros(n, m % 2)], 1).to(torch.int64) & 15
    return (q[:, 0::2] | q[:, 1::2] << 4).to(torch.uint8), scale


def load(q, scale, kind, block, values, dtype):
    if kind == "int4":
        b = q.to(torch.int64)
        q = torch.stack([b & 15, b >> 4], -1).reshape(b.shape[0], -1)[:, :values]
        q = q - 16 * (q >= 8)
    return (q.float() * scale.repeat_interleave(block, 1)[:, :values]).to(dtype)
