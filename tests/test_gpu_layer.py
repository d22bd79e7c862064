"""The layer operators on the GPU against their plain 64-bit forms (tests/layer_ref.py).

Tolerances: an output is rounded once to its type (half a step of it), and the fp32 computation before
that makes at most `count` roundings of 2^-24 relative to the magnitude of the terms it sums. Counts
are worst cases: a recurrence over L tokens multiplies by L decays, each off by the exp2's argument
rounding (an argument of at most 30 in magnitude before the decay is negligible, two roundings: 60) and
by its result (2), on top of the products and sums of each token."""
import pytest
import torch

import state_space_sequence_mamba3_amd as m3
from tests import layer_ref as R
from tests.gpu_util import device, note

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rand(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(dtype)


def up(t):
    return t.to(device()) if t is not None else None


# 700 sequences of 0 to about 10 tokens
MANY = [0] + sorted(torch.randint(0, 901, (699,), generator=torch.Generator().manual_seed(7)).tolist()) + [900]

# ----------------------------------------------------------------------------- convolution
CONV = [  # batch, seqlen, dim, width, cu
    (2, 37, 64, 4, None), (1, 1, 8, 4, None), (3, 2, 40, 4, None), (1, 130, 1, 2, None), (2, 19, 7, 3, None),
    (1, 70, 24, 8, None), (2, 33, 512, 5, None), (1, 100, 72, 4, [0, 0, 1, 3, 3, 40, 41, 100, 100]),
    (0, 9, 16, 4, None), (1, 900, 8, 4, MANY), (1, 64, 13, 6, [0, 2, 64]), (1, 5, 16, 7, [0, 1, 2, 3, 4, 5]), (1, 0, 8, 4, [0, 0, 0]), (2, 0, 8, 4, None),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", CONV)
@pytest.mark.parametrize("full", [True, False])
def test_conv(case, dtype, full):
    b, L, D, W, cu = case
    note(f"conv {case} {dtype} full={full}")
    g = gen(11 + L + D + W)
    S = len(cu) - 1 if cu else b
    x, w = rand(g, b, L, D, dtype=dtype), rand(g, D, W, std=0.5)
    bias = rand(g, D, std=0.5) if full else None
    cin = rand(g, S, W - 1, D, dtype=dtype) if full else None
    dy, dco = rand(g, b, L, D, dtype=dtype), rand(g, S, W - 1, D, dtype=dtype) if full else None
    cut = torch.tensor(cu, dtype=torch.int32) if cu else None
    ref = R.conv(x, w, bias, full, cin, cu, dy, dco)
    mag = R.conv(x, w, bias, full, cin, cu, dy, dco, mag=True)
    y, co = m3.mamba3_conv_fwd(up(x), up(w), up(bias), silu=full, conv_in=up(cin), cu_seqlens=up(cut))
    # W products and sums, then exp, reciprocal and two products
    R.check(y, ref["y"], mag["y"], W + 12, "y")
    assert torch.equal(co.cpu().double(), ref["conv_out"]), "conv_out"
    gr = m3.mamba3_conv_bwd(up(x), up(w), up(bias), dy=up(dy), dconv_out=up(dco), silu=full, conv_in=up(cin),
                            cu_seqlens=up(cut))
    assert set(gr) == {"dx", "dweight"} | ({"dbias", "dconv_in"} if full else set())
    n = b * L
    for k, count in (("dx", 2 * W + 24), ("dweight", n + W + 24), ("dbias", n + W + 24), ("dconv_in", 2 * W + 24)):
        if k in gr:
            R.check(gr[k], ref[k], mag[k], count, k)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_conv_views_and_steps(dtype):
    """x as the half of a wider row; a prompt's state taken up by single tokens through slots equals the
    convolution of the whole, and rows without a slot stay as they were."""
    g = gen(5)
    b, L, D, W = 3, 21, 64, 4
    wide = rand(g, b, L, 2 * D + 8, dtype=dtype)
    w, bias = rand(g, D, W, std=0.5), rand(g, D, std=0.5)
    view = up(wide)[:, :, D:2 * D]
    whole, _ = m3.mamba3_conv_fwd(view.contiguous(), up(w), up(bias))
    y, _ = m3.mamba3_conv_fwd(view, up(w), up(bias))
    assert torch.equal(y, whole)
    n = 13
    y0, state = m3.mamba3_conv_fwd(view[:, :n].contiguous(), up(w), up(bias))
    assert torch.equal(y0, whole[:, :n])
    pool = torch.full((7, W - 1, D), 9.0, dtype=dtype, device=device())
    slots = torch.tensor([5, -1, 0, 2, 7], dtype=torch.int32, device=device())
    rows = torch.tensor([0, 0, 1, 2, 0], device=device())
    for r, s in ((0, 5), (1, 0), (2, 2)):
        pool[s] = state[r]
    for t in range(n, L):
        xt = view[:, t][rows]
        yt = torch.full((5, D), 3.0, dtype=dtype, device=device())
        m3.mamba3_conv_step(xt, up(w), up(bias), conv=pool, slots=slots, y=yt)
        assert torch.equal(yt[[0, 2, 3]], whole[:, t]), t
        assert bool((yt[[1, 4]] == 3.0).all())
    assert bool((pool[[1, 3, 4, 6]] == 9.0).all())
    assert torch.equal(pool[[5, 0, 2]], view[:, L - W + 1:])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim", [3, 4, 5, 7, 9, 15, 65, 255, 257, 259, 511, 513, 1025])
def test_conv_rows_of_any_length(dim, dtype):
    """Channel counts around the pieces and workgroups that a row is cut into, rows that start at any
    element: the last pieces of a row share channels."""
    note(f"conv rows {dim} {dtype}")
    g = gen(900 + dim)
    L, W = 70, 4
    cu = [0, 33, 34, L]
    wide = rand(g, 1, L, 2 * dim + 1, dtype=dtype)
    x, dy = wide[:, :, :dim], wide[:, :, dim + 1:]
    w, bias = rand(g, dim, W, std=0.5), rand(g, dim, std=0.5)
    cin, dco = rand(g, 3, W - 1, dim, dtype=dtype), rand(g, 3, W - 1, dim, dtype=dtype)
    ref = R.conv(x, w, bias, True, cin, cu, dy, dco)
    mag = R.conv(x, w, bias, True, cin, cu, dy, dco, mag=True)
    cut, on = up(torch.tensor(cu, dtype=torch.int32)), up(wide)
    xd, dyd = on[:, :, :dim], on[:, :, dim + 1:]
    # outputs one element behind an aligned address, a guard on both sides
    y = torch.full((L * dim + 2,), 5.0, dtype=dtype, device=device())
    m3.mamba3_conv_fwd(xd, up(w), up(bias), conv_in=up(cin), cu_seqlens=cut, y=y[1:-1].view(1, L, dim))
    R.check(y[1:-1].view(1, L, dim), ref["y"], mag["y"], W + 12, "y")
    assert float(y[0]) == 5.0 and float(y[-1]) == 5.0
    gr = m3.mamba3_conv_bwd(xd, up(w), up(bias), dy=dyd, dconv_out=up(dco), conv_in=up(cin), cu_seqlens=cut)
    for k, count in (("dx", 2 * W + 24), ("dweight", L + W + 24), ("dbias", L + W + 24), ("dconv_in", 2 * W + 24)):
        R.check(gr[k], ref[k], mag[k], count, k)


# ----------------------------------------------------------------------------- selective scan
SCAN = [  # batch, seqlen, dim, N, G, cu
    (2, 37, 64, 16, 1, None), (1, 1, 8, 16, 1, None), (2, 16, 100, 16, 1, None), (1, 33, 1, 1, 1, None),
    (1, 50, 130, 4, 2, None), (2, 17, 36, 8, 3, None), (1, 65, 48, 24, 2, None), (1, 40, 20, 64, 1, None),
    (1, 31, 12, 128, 1, None), (1, 29, 15, 7, 3, None), (1, 23, 10, 50, 2, None), (1, 20, 6, 100, 2, None),
    (1, 90, 72, 16, 1, [0, 0, 1, 3, 3, 40, 41, 90, 90]), (1, 34, 9, 13, 1, [0, 17, 17, 34]),
    (1, 0, 8, 16, 1, [0, 0, 0]), (2, 0, 8, 16, 1, None),
    # long enough to run as segments, and enough sequences not to
    (1, 300, 40, 16, 1, None), (3, 200, 9, 16, 1, None), (2, 129, 36, 24, 2, None), (1, 150, 8, 128, 1, None),
    (1, 400, 20, 16, 1, [0, 0, 64, 65, 65, 300, 399, 400]), (1, 333, 6, 5, 2, [0, 200, 333]),
    (64, 70, 256, 16, 1, None), (0, 9, 8, 16, 1, None), (1, 900, 8, 16, 1, MANY),
    # fewer than four states
    (2, 90, 40, 1, 1, None), (1, 90, 70, 2, 2, None), (1, 400, 40, 3, 1, [0, 100, 101, 400]), (2, 19, 12, 3, 3, None),
]


def scan_inputs(case, dtype, full, seed=0):
    b, L, D, N, G, cu = case
    g = gen(100 * seed + 31 + L + D + N)
    S = len(cu) - 1 if cu else b
    a = dict(x=rand(g, b, L, D, dtype=dtype), dt=rand(g, b, L, D, dtype=dtype, std=0.7),
             A=-torch.exp(rand(g, D, N, std=0.7)), B=rand(g, b, L, G, N, dtype=dtype), C=rand(g, b, L, G, N, dtype=dtype),
             D=rand(g, D) if full else None)
    if not full:
        a["dt"] = a["dt"].abs()
    kw = dict(z=rand(g, b, L, D, dtype=dtype, std=2.0) if full else None,
              dt_bias=rand(g, D) - 2 if full else None, dt_softplus=full,
              h_in=rand(g, S, D, N) if full else None)
    dy, dho = rand(g, b, L, D, dtype=dtype), rand(g, S, D, N) if full else None
    return a, kw, dy, dho, torch.tensor(cu, dtype=torch.int32) if cu else None


def scan_ref(a, kw, cu, dy=None, dho=None, mag=False):
    return R.scan(a["x"], a["dt"], a["A"], a["B"], a["C"], a["D"], kw["z"], kw["dt_bias"], kw["dt_softplus"],
                  kw["h_in"], cu, dy, dho, mag=mag)


def dev(d):
    return {k: up(v) if isinstance(v, torch.Tensor) else v for k, v in d.items()}


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", SCAN)
@pytest.mark.parametrize("full", [True, False])
def test_selective_scan(case, dtype, full):
    note(f"selective scan {case} {dtype} full={full}")
    a, kw, _, _, cu = scan_inputs(case, dtype, full)
    L, N = case[1], case[3]
    ref, mag = scan_ref(a, kw, case[5]), scan_ref(a, kw, case[5], mag=True)
    y, h = m3.mamba3_selective_scan_fwd(**dev(a), **dev(kw), cu_seqlens=up(cu))
    R.check(h, ref["h_out"], mag["h_out"], 70 * L + 16, "h_out")
    R.check(y, ref["y"], mag["y"], 70 * L + N + 32, "y")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", SCAN)
@pytest.mark.parametrize("full", [True, False])
def test_selective_scan_bwd(case, dtype, full):
    note(f"selective scan backward {case} {dtype} full={full}")
    a, kw, dy, dho, cu = scan_inputs(case, dtype, full)
    b, L, D, N, G, _ = case
    ref = scan_ref(a, kw, case[5], dy, dho)
    mag = scan_ref(a, kw, case[5], dy, dho, mag=True)
    gr = m3.mamba3_selective_scan_bwd(**dev(a), **dev(kw), dy=up(dy), dh_out=up(dho), cu_seqlens=up(cu))
    assert set(gr) == {"dx", "ddt", "dB", "dC", "dA"} | ({"dD", "dz", "ddt_bias", "dh_in"} if full else set())
    # both the states and the carried gradient make the recurrence's roundings
    steps = 140 * L + 64
    for k in gr:
        extra = D if k in ("dB", "dC") else b * L if k in ("dA", "dD", "ddt_bias") else N
        R.check(gr[k], ref[k], mag[k], steps + extra, k)
    again = m3.mamba3_selective_scan_bwd(**dev(a), **dev(kw), dy=up(dy), dh_out=up(dho), cu_seqlens=up(cu))
    for k in gr:
        assert torch.equal(gr[k], again[k]), k


def test_selective_scan_bwd_differences():
    """The gradient against central differences of the 64-bit forward, in a random direction of every
    input: the difference quotient of step e is off by O(e^2) and the gradient by fp32's roundings."""
    case = (1, 24, 12, 16, 2, [0, 5, 24])
    a, kw, dy, dho, cu = scan_inputs(case, F32, True)
    gr = m3.mamba3_selective_scan_bwd(**dev(a), **dev(kw), dy=up(dy), dh_out=up(dho), cu_seqlens=up(cu))
    both = {**a, **kw}
    names = dict(dx="x", ddt="dt", dB="B", dC="C", dA="A", dD="D", dz="z", ddt_bias="dt_bias", dh_in="h_in")

    def loss(v):
        v = dict(v)
        r = R.scan(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], v["z"], v["dt_bias"], True, v["h_in"], case[5])
        return float((r["y"] * dy).sum() + (r["h_out"] * dho).sum())

    g = gen(77)
    for k, name in names.items():
        way = torch.randn(both[name].shape, generator=g).double()
        e = 1e-4
        lo, hi = (loss({**both, name: both[name].double() + s * e * way}) for s in (-1, 1))
        want = (hi - lo) / (2 * e)
        terms = gr[k].cpu().double() * way
        got = float(terms.sum())
        # e^2 / 6 times a third derivative of the order of the terms' sum (a few hundred times, at worst)
        assert abs(got - want) <= 2e-5 * float(terms.abs().sum()), (k, got, want)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", [(2, 29, 64, 16, 1, None), (1, 20, 48, 24, 2, None), (1, 18, 9, 13, 1, None),
                                  (2, 17, 12, 128, 1, None),
                                  (2, 18, 36, 3, 2, None), (1, 18, 8, 1, 1, None), (1, 18, 40, 18, 1, None)])
def test_selective_steps_continue_a_prompt(case, dtype):
    """A prompt's state taken up by single tokens through slots; inputs as views of wider rows."""
    note(f"selective steps {case} {dtype}")
    b, L, D, N, G, _ = case
    a, kw, _, _, _ = scan_inputs(case, dtype, True, seed=3)
    ref, mag = scan_ref(a, kw, None), scan_ref(a, kw, None, mag=True)
    da, dk = dev(a), dev(kw)
    n = L - 6
    cut = lambda t, lo, hi: t[:, lo:hi].contiguous()   # noqa: E731
    toks = {k: da[k] for k in ("x", "dt", "B", "C")}
    y0, h = m3.mamba3_selective_scan_fwd(**{**da, **{k: cut(v, 0, n) for k, v in toks.items()}},
                                         **{**dk, "z": cut(dk["z"], 0, n)})
    R.check(y0, ref["y"][:, :n], mag["y"][:, :n], 70 * L + N + 32, "prompt")
    pool = torch.full((2 * b + 3, D, N), 5.0, device=device())
    slots = torch.tensor([2 * i + 1 for i in range(b)] + [-1, 2 * b + 3], dtype=torch.int32, device=device())
    pool[slots[:b].long()] = h
    rows = torch.tensor(list(range(b)) + [0, 0], device=device())
    # one wide row a token, as a projection leaves it: z, x, dt, B, C side by side
    for t in range(n, L):
        parts = [dk["z"][:, t], da["x"][:, t], da["dt"][:, t], da["B"][:, t].reshape(b, -1), da["C"][:, t].reshape(b, -1)]
        row = torch.cat(parts, 1)[rows]
        z, x, dt, B, C = row.split([D, D, D, G * N, G * N], 1)
        y = torch.full((b + 2, D), 3.0, dtype=dtype, device=device())
        m3.mamba3_selective_step(x, dt, da["A"], B.unflatten(1, (G, N)), C.unflatten(1, (G, N)), da["D"], h=pool, z=z,
                                 dt_bias=dk["dt_bias"], dt_softplus=True, slots=slots, y=y)
        R.check(y[:b], ref["y"][:, t], mag["y"][:, t], 70 * L + N + 32, f"step {t}")
        assert bool((y[b:] == 3.0).all())
    R.check(pool[slots[:b].long()], ref["h_out"], mag["h_out"], 70 * L + 16, "state")
    rest = [i for i in range(2 * b + 3) if i not in slots[:b].tolist()]
    assert bool((pool[rest] == 5.0).all())


@pytest.mark.parametrize("case", [(64, 20, 256, 16, 1, None), (2, 300, 24, 16, 1, None), (1, 300, 24, 16, 1, [0, 100, 300])])
def test_selective_scan_state_in_place(case):
    """h_out = h_in, in one pass and in segments."""
    a, kw, _, _, cu = scan_inputs(case, F32, True, seed=5)
    a, kw = dev(a), dev(kw)
    y, h = m3.mamba3_selective_scan_fwd(**a, **kw, cu_seqlens=up(cu))
    own = kw["h_in"].clone()
    y2, h2 = m3.mamba3_selective_scan_fwd(**a, **{**kw, "h_in": own}, h_out=own, cu_seqlens=up(cu))
    assert h2 is own and torch.equal(y, y2) and torch.equal(h, own)


def test_selective_scan_views():
    """x and z as the halves of one projection, B and C as slices of another, equal dense inputs."""
    g = gen(9)
    for D, N in ((64, 16), (21, 5)):
        xz = up(rand(g, 2, 19, 2 * D + 3, dtype=BF16))
        bc = up(rand(g, 2, 19, 2 * N + D, dtype=BF16))
        A = up(-torch.exp(rand(g, D, N)))
        x, z, dt = xz[:, :, 3:3 + D], xz[:, :, 3 + D:], bc[:, :, 2 * N:].abs()
        dt = torch.cat([dt, dt], 2)[:, :, :D]       # (a strided view again)
        B, C = bc[:, :, :N].unflatten(2, (1, N)), bc[:, :, N:2 * N].unflatten(2, (1, N))
        dy = up(rand(g, 2, 19, D + 1, dtype=BF16))[:, :, 1:]
        one = m3.mamba3_selective_scan_fwd(x, dt, A, B, C, z=z)
        two = m3.mamba3_selective_scan_fwd(*(t.contiguous() for t in (x, dt, A, B, C)), z=z.contiguous())
        assert all(torch.equal(p, q) for p, q in zip(one, two))
        one = m3.mamba3_selective_scan_bwd(x, dt, A, B, C, z=z, dy=dy)
        two = m3.mamba3_selective_scan_bwd(*(t.contiguous() for t in (x, dt, A, B, C)), z=z.contiguous(),
                                           dy=dy.contiguous())
        assert all(torch.equal(one[k], two[k]) for k in two)


def test_selective_scan_extremes():
    """Steps that forget everything (exp underflows to 0) and steps of 0, large and tiny softplus inputs."""
    g = gen(4)
    D, N, L = 16, 16, 40
    a, kw, _, _, _ = scan_inputs((1, L, D, N, 1, None), F32, True, seed=8)
    a["dt"][0, 5] = 90.0            # softplus of 90 is 90: exp(-90 |A|) is 0 or nearly
    a["dt"][0, 6:9] = -100.0        # a step of 4e-44: the state stays
    a["dt"][0, 20] = 20.0 + 2.0     # the border of softplus' second form, with the bias
    a["A"][:, 3] = -80.0
    a["A"][:, 4] = 0.0
    ref, mag = scan_ref(a, kw, None), scan_ref(a, kw, None, mag=True)
    y, h = m3.mamba3_selective_scan_fwd(**dev(a), **dev(kw))
    R.check(h, ref["h_out"], mag["h_out"], 70 * L + 16, "h_out")
    R.check(y, ref["y"], mag["y"], 70 * L + N + 32, "y")


# ----------------------------------------------------------------------------- RMS norm
NORM = [(1, 1), (5, 64), (3, 40), (7, 513), (4, 1000), (2, 2048), (2100, 1024), (2050, 2000), (3, 4100), (2, 8192),
        (2, 8200), (3, 9001), (4500, 200), (0, 64), (0, 9000)]


def norm_inputs(rows, dim, dtype, rt, seed=0):
    g = gen(rows + dim + seed)
    res = rand(g, rows, dim, dtype=rt, std=3.0) if rt is not None else None
    return rand(g, rows, dim, dtype=dtype), res, rand(g, dim) + 1.0, g


@pytest.mark.parametrize("types", [(F32, F32), (BF16, F32), (BF16, BF16), (BF16, None)])
@pytest.mark.parametrize("rows,dim", NORM)
def test_rmsnorm(rows, dim, types):
    note(f"rmsnorm {rows}x{dim} {types}")
    x, res, w, _ = norm_inputs(rows, dim, *types)
    s, v = R.norm(x, res, w, 1e-5)
    got = m3.mamba3_rmsnorm_fwd(up(x), up(w), residual=up(res), eps=1e-5)
    assert set(got) == {"y"} | ({"residual"} if res is not None else set())
    # the sum of dim squares (each of them positive: its relative error is at most dim + 2 roundings, half
    # of that after the root), rsqrt, two products, the residual's sum
    mag = (x.double().abs() + (res.double().abs() if res is not None else 0)) * (v / s).nan_to_num()
    R.check(got["y"], v, mag, dim + 10, "y")
    if res is not None:
        R.check(got["residual"], s, s, 1, "residual")


@pytest.mark.parametrize("rows,dim", NORM)
@pytest.mark.parametrize("qblock", [0, 32, 128, 256])
@pytest.mark.parametrize("quant", ["e4m3", "int8"])
def test_rmsnorm_quantised(rows, dim, qblock, quant):
    x, res, w, _ = norm_inputs(rows, dim, BF16, BF16)
    x[:1] = 0
    res[:1] = 0                                      # a row of zeros
    note(f"rmsnorm {quant} {rows}x{dim} block {qblock}")
    _, v = R.norm(x, res, w, 1e-5)
    got = m3.mamba3_rmsnorm_fwd(up(x), up(w), residual=up(res), eps=1e-5, want_y=False, quant=quant, qblock=qblock)
    assert set(got) == {"q", "scale", "residual"}
    block = dim if qblock == 0 else qblock
    blocks = -(-dim // block)
    pad = torch.nn.functional.pad(v, (0, blocks * block - dim)).view(rows, blocks, block)
    top = 448.0 if quant == "e4m3" else 127.0
    want = (pad.abs().amax(-1) / top).clamp(min=2.0 ** -126)
    assert got["scale"].shape == want.shape
    R.check(got["scale"], want, want, dim + 12, "scale")
    scale = got["scale"].cpu().double().repeat_interleave(block, 1)[:, :dim]
    q = got["q"].cpu().double()
    # the nearest 8-bit value of v / scale, off by v's own error before the rounding
    ideal = v / scale
    err = (dim + 14) * R.U32 * ideal.abs()
    if quant == "e4m3":
        # half a step: 2^-4 relative, 2^-10 below the smallest normal value 2^-6
        half = torch.maximum(ideal.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10).double())
    else:
        half = torch.tensor(0.5).double()
    assert bool(((q - ideal).abs() <= half * (1 + 1e-6) + err * 2).all())
    assert bool((q.abs() <= top).all())
    assert bool((q[:1] == 0).all())


def test_rmsnorm_in_place_views_and_both_outputs():
    g = gen(2)
    wide, res, w = up(rand(g, 6, 3, 80, dtype=BF16)), up(rand(g, 6, 3, 64)), up(rand(g, 64) + 1)
    x = wide[:, :, 8:72]
    keep = res.clone()
    got = m3.mamba3_rmsnorm_fwd(x, w, residual=res, residual_out=res, quant="e4m3", qblock=32)
    assert got["residual"] is res and torch.equal(res, x.float() + keep)
    other = m3.mamba3_rmsnorm_fwd(x.contiguous(), w, residual=keep)
    assert torch.equal(got["y"], other["y"]) and got["scale"].shape == (6, 3, 2)
    alone = m3.mamba3_rmsnorm_fwd(x, w, residual=keep, want_y=False, quant="e4m3", qblock=32)
    assert torch.equal(alone["q"].view(torch.uint8), got["q"].view(torch.uint8))


def test_rmsnorm_first_layer():
    """A residual stream begun: residual_out without a residual is x in its type."""
    x, _, w, _ = norm_inputs(6, 72, BF16, None)
    out = torch.empty(6, 72, device=device())
    got = m3.mamba3_rmsnorm_fwd(up(x), up(w), residual_out=out)
    assert got["residual"] is out and torch.equal(out.cpu(), x.float())
    assert torch.equal(got["y"], m3.mamba3_rmsnorm_fwd(up(x), up(w))["y"])


@pytest.mark.parametrize("types", [(F32, F32), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("rows,dim", NORM)
@pytest.mark.parametrize("carry", [True, False])
def test_rmsnorm_bwd(rows, dim, types, carry):
    note(f"rmsnorm backward {rows}x{dim} {types} carry={carry}")
    dtype, rt = types
    dy, s, w, g = norm_inputs(rows, dim, dtype, rt, seed=7)
    dres = rand(g, rows, dim, dtype=rt) if carry else None
    ref, mag = R.norm_bwd(s, w, dy, dres, 1e-5), R.norm_bwd(s, w, dy, dres, 1e-5, mag=True)
    got = m3.mamba3_rmsnorm_bwd(up(s), up(w), dy=up(dy), dresidual_out=up(dres), eps=1e-5)
    assert set(got) == {"dx", "dresidual", "dweight"}
    R.check(got["dresidual"], ref[0], mag[0], 4 * dim + 32, "dresidual")
    R.check(got["dx"], ref[0], mag[0], 4 * dim + 32, "dx")
    R.check(got["dweight"], ref[1], mag[1], rows + dim + 16, "dweight")
    again = m3.mamba3_rmsnorm_bwd(up(s), up(w), dy=up(dy), dresidual_out=up(dres), eps=1e-5)
    assert all(torch.equal(got[k], again[k]) for k in got)


def test_rmsnorm_not_finite():
    """A NaN or an infinity stays in its row; the block that holds it shows it in its scale."""
    x = torch.ones(4, 256)
    x[1, 3], x[2, 200] = float("nan"), float("inf")
    for quant in (None, "e4m3"):
        got = m3.mamba3_rmsnorm_fwd(up(x), quant=quant, qblock=128)
        assert bool(torch.isfinite(got["y"][[0, 3]]).all())
        assert bool(torch.isnan(got["y"][1]).all())
        # an infinite row: its finite values become 0, the infinite one has no value
        assert bool(torch.isnan(got["y"][2, 200])) and bool((got["y"][2, :200] == 0).all())
        if quant:
            assert bool(torch.isfinite(got["scale"][[0, 3]]).all()) and bool(torch.isnan(got["scale"][1]).all())
