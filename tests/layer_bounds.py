"""Roundings that the layer operators' fp32 computations make, counted along their sums and recurrences
instead of by their lengths, for the tests that hold them close: an error of one part in a few thousand
(a value rounded to bf16 on the way) lies outside."""
import torch


def norm_depth(dim):
    """Additions on the longest path of a row's sum: a lane adds pieces of 8 values (two at least where a
    wave has a row, one for every 2048 values of a long row), then 6 levels over the wave, then up to 16
    waves one by one."""
    return 8 * max(2, -(-dim // 2048)) + 6 + 16


def rms_count(dim):
    """Roundings of 1 / sqrt(mean s^2 + eps): s itself and its square (3), the sum, the division and eps (2),
    halved by the root; the root's own unit in the last place (2) and a power of two."""
    return (norm_depth(dim) + 5) // 2 + 3


def norm_count(dim):
    """Of v = s r w, s rounded once, relative to v."""
    return rms_count(dim) + 3


def norm_bwd_count(dim):
    """Of dres + r (w dy - sh mean(w dy sh)), relative to the terms' magnitudes: sh has r's and one more; the
    mean has two products a value, the sum, r and two more; then three products and two sums."""
    return (rms_count(dim) + 1) + (2 + norm_depth(dim) + rms_count(dim) + 2) + rms_count(dim) + 5


def dweight_count(rows, dim):
    """Of the sum over rows of dy sh: r and two products, then the rows that a workgroup walks (256
    workgroups at least, or all rows by four waves above 8192 values), then what is left of at most 1024
    workgroups by 16 threads each."""
    walked = rows // 4 + 1 if dim > 8192 else rows // 256 + 1
    return rms_count(dim) + 2 + walked + 3 + 1024 // 16 + 16


def scan(x, dt, A, B, C, D, z, bias, softplus, h_in, cu, dy, dh_out, window, spoil=None):
    """The selective scan and its gradients in 64 bits, token by token, with a bound on the error of an fp32
    computation of each: name -> (value, error in units of 2^-24 of what it is off by).

    Every product, sum, exp2, log2 and reciprocal is off by one rounding (2 for the last three) of its result; a
    decay exp(s A) by |s A| times what s and the exponent's two products are off by, and, because
    states are carried over segments by the exponential of a sum of at most `window` steps, by |A| times
    what that sum has so far. Errors of a state run through its own recurrence: decays shrink them.
    `spoil(which, token, value)` may change the state that enters a token ("h") or the gradient that leaves it
    ("g"): a planted mistake."""
    spoil = spoil or (lambda what, t, v: v)
    lead, dim, (G, N) = x.shape[:2], x.shape[2], B.shape[2:]
    fl = lambda t: t.double().reshape(-1, *t.shape[2:])   # noqa: E731
    of = torch.arange(dim) // (dim // G)
    xd, Bd, Cd, Ad, rd = fl(x), fl(B), fl(C), A.double(), fl(dy)
    raw = fl(dt) + (bias.double() if bias is not None else 0)
    s = torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw
    # w = e^raw by raw's rounding, the product with log2 e (2) and exp2; log(1 + w) by log2, the product and
    # the correction; 1 / (1 + e^-raw) by the same exponent, a sum and a reciprocal
    ks = 3 * raw.abs() + 8 if softplus else torch.ones_like(raw)
    kg = 3 * raw.abs() + 6
    gate = 1 / (1 + torch.exp(-raw)) if softplus else torch.ones_like(raw)
    Dd = D.double() if D is not None else torch.zeros(dim).double()
    if z is not None:
        zd = fl(z)
        sg = 1 / (1 + torch.exp(-zd))
        sil, kz, ksig = zd * sg, 2 * zd.abs() + 8, 2 * zd.abs() + 5
        dsil, dterms = sg + zd * sg * (1 - sg), sg + zd.abs() * sg * (1 - sg)
        edsil = sg * ksig + zd.abs() * sg * (2 * ksig + 4) + 2 * dterms
        r, kr = rd * sil, kz + 1
    else:
        sil, r, kr = torch.ones_like(rd), rd, torch.zeros_like(rd)
        kz = kr
    T = xd.shape[0]
    v = {k: torch.zeros(T, dim).double() for k in ("y", "dx", "ddt", "dz")}
    v.update({k: torch.zeros(T, G, N).double() for k in ("dB", "dC")})
    e = {k: t.clone() for k, t in v.items()}
    for k, shape in dict(dA=(dim, N), dD=(dim,), ddt_bias=(dim,)).items():
        v[k], e[k] = torch.zeros(shape).double(), torch.zeros(shape).double()
    ends, dins = [], []
    at = [int(c) for c in cu] if cu is not None else [i * lead[1] for i in range(lead[0] + 1)]
    group = lambda t: t.view(G, -1, N).sum(1)   # noqa: E731
    for i, (t0, t1) in enumerate(zip(at[:-1], at[1:])):
        n = t1 - t0
        h = h_in[i].double() if h_in is not None else torch.zeros(dim, N).double()
        hm, he = h.abs(), torch.zeros(dim, N).double()
        run = torch.cat([torch.zeros(1, dim).double(), s[t0:t1].abs().cumsum(0)])
        kept = []
        for t in range(t0, t1):
            k = t - t0
            near = run[k + 1] - run[max(0, k + 1 - window)]         # the sum of the last steps
            a = torch.exp(s[t][:, None] * Ad)
            ea = (s[t][:, None] * Ad).abs() * (ks[t][:, None] + 4) + near[:, None] * Ad.abs() + 2
            h = spoil("h", k, h)
            kept.append((h, hm, he, a, ea))
            u = (s[t] * xd[t])[:, None] * Bd[t][of]
            he = a * he + a * hm * (ea + 1) + u.abs() * (ks[t][:, None] + 3)
            h, hm = a * h + u, a * hm + u.abs()
            he = he + hm
            c = Cd[t][of]
            ym, ye = (hm * c.abs()).sum(-1) + (Dd * xd[t]).abs(), (he * c.abs()).sum(-1)
            ye = ye + (N + 4) * ym
            y0 = (h * c).sum(-1) + Dd * xd[t]
            v["y"][t], e["y"][t] = y0 * sil[t], ye * sil[t].abs() + ym * sil[t].abs() * (kz[t] + 1)
            kept[-1] += (h, hm, he, y0, ym, ye)
        ends.append((h, he))
        q = dh_out[i].double() if dh_out is not None else torch.zeros(dim, N).double()
        qm, qe = q.abs(), torch.zeros(dim, N).double()
        for t in range(t1 - 1, t0 - 1, -1):
            k = t - t0
            hp, hpm, hpe, a, ea, h, hm, he, y0, ym, ye = kept[k]
            b, c, st, xt, rt = Bd[t][of], Cd[t][of], s[t][:, None], xd[t], r[t][:, None]
            q = spoil("g", k, q)
            g, gm = q + rt * c, qm + (rt * c).abs()
            ge = qe + (rt * c).abs() * (kr[t][:, None] + 1) + gm
            if z is not None:
                v["dz"][t] = rd[t] * y0 * dsil[t]
                e["dz"][t] = rd[t].abs() * (ye * dterms[t] + ym * edsil[t])
            v["dC"][t] = group(rt * h)
            e["dC"][t] = group(rt.abs() * he + rt.abs() * hm * (kr[t][:, None] + 1 + dim // G))
            u, um = (st * xt[:, None]), (st * xt[:, None]).abs()
            v["dB"][t] = group(g * u)
            e["dB"][t] = group(ge * um + gm * um * (ks[t][:, None] + 2 + dim // G))
            du, dum, due = (g * b).sum(-1), (gm * b.abs()).sum(-1), (ge * b.abs()).sum(-1)
            due = due + (N + 3) * dum
            q, qm, qe = g * a, gm * a, a * ge + a * gm * (ea + 1)
            w, wm, we = q * hp, qm * hpm, qe * hpm + qm * hpe + qm * hpm
            v["dA"] += w * st
            e["dA"] += we * st.abs() + wm * st.abs() * (ks[t][:, None] + 1 + n)
            ds, dsm = du * xt + (w * Ad).sum(-1), dum * xt.abs() + (wm * Ad.abs()).sum(-1)
            dse = due * xt.abs() + (we * Ad.abs()).sum(-1) + (N + 4) * dsm
            v["ddt"][t], e["ddt"][t] = ds * gate[t], dse * gate[t] + dsm * gate[t] * (kg[t] + 1)
            v["ddt_bias"] += v["ddt"][t]
            e["ddt_bias"] += e["ddt"][t] + dsm * gate[t] * n
            v["dx"][t] = du * s[t] + Dd * r[t]
            e["dx"][t] = due * s[t].abs() + dum * s[t].abs() * (ks[t] + 2) + (Dd * r[t]).abs() * (kr[t] + 3)
            v["dD"] += r[t] * xt
            e["dD"] += (r[t] * xt).abs() * (kr[t] + 2 + n)
        dins.append((q, qe))
    for k in ("y", "dx", "ddt", "dz"):
        v[k], e[k] = v[k].view(x.shape), e[k].view(x.shape)
    for k in ("dB", "dC"):
        v[k], e[k] = v[k].view(B.shape), e[k].view(B.shape)
    for k, rows in (("h_out", ends), ("dh_in", dins)):
        v[k], e[k] = torch.stack([a for a, _ in rows]), torch.stack([b for _, b in rows])
    # sums over sequences and segments
    for k in ("dA", "dD", "ddt_bias"):
        e[k] += (len(ends) + T // window + 2) * v[k].abs()
    return {k: (v[k], e[k]) for k in v}


def off(got, want):
    """How far `got` is from want = (value, error in units of 2^-24), over what it may be: the output's own
    rounding, and the error (1 % for products of errors)."""
    v, e = want
    half = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float64 else 0.0
    room = half * v.abs() * 1.001 + 1.01 * 2.0 ** -24 * e * (1 + half) + 1e-37
    return float(((got.detach().cpu().double() - v).abs() / room).max()) if v.numel() else 0.0


def scan_case(b, L, dim, N, G, cu, seed, positive, dtype=torch.float32, plain=False):
    """Inputs of a scan of slow decays (e^-0.02 a token for the middle state, with steps around 0.05), so that a state
    lives for several segments of 64 tokens. `positive`: no sum cancels, which makes the bounds relative;
    `plain`: no softplus, gate and bias."""
    g = torch.Generator().manual_seed(seed)
    S = len(cu) - 1 if cu else b
    normal = lambda *shape: torch.randn(shape, generator=g)   # noqa: E731
    r = (lambda *shape: normal(*shape).abs()) if positive else normal
    dt = 0.05 + 0.03 * torch.rand((b, L, dim), generator=g) if plain else 0.3 * normal(b, L, dim) - 3
    return dict(x=r(b, L, dim).to(dtype), dt=dt.to(dtype), A=-0.4 * torch.exp(0.5 * normal(dim, N)), B=r(b, L, G, N).to(dtype),
                C=r(b, L, G, N).to(dtype), D=r(dim), z=None if plain else (1.5 * r(b, L, dim)).to(dtype),
                bias=None if plain else 0.2 * normal(dim), softplus=not plain, h_in=4 * r(S, dim, N), cu=cu,
                dy=r(b, L, dim).to(dtype), dh_out=4 * r(S, dim, N))
