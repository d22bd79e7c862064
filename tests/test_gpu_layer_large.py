"""Layer operators at sizes whose arrays and pools pass 2^31 and 2^32 elements, and with sequence bounds outside the
batch."""
import pytest
import torch

import state_space_sequence_mamba3_amd as m3
from tests import layer_bounds as LB
from tests import layer_ref as R
from tests.gpu_util import device, note
from tests.test_gpu_layer import BF16, dev, gen, rand, scan_inputs, up

pytestmark = pytest.mark.gpu


def test_selective_scan_of_a_long_sequence():
    """More than 2^31 values of B and of C: the first tokens, and the last ones of a state that has forgotten what
    lies 300 tokens back (decays of e^-0.3 a token at least), equal the 64-bit form."""
    L, D, N, n = (1 << 25) + 77, 4, 64, 200
    note(f"scan of {L} tokens, B and C {L * N * 2 >> 20} MiB each")
    g = torch.Generator(device=device()).manual_seed(3)
    x, dt = (torch.randn((1, L, D), generator=g, device=device(), dtype=BF16) for _ in range(2))
    B, C = (torch.randn((1, L, 1, N), generator=g, device=device(), dtype=BF16) for _ in range(2))
    A, skip, bias = -1 - rand(gen(1), D, N).abs(), rand(gen(2), D), torch.full((D,), 3.0)
    y, h = m3.mamba3_selective_scan_fwd(x, dt.clamp(min=-3.5), up(A), B, C, up(skip), dt_bias=up(bias), dt_softplus=True)
    for a, lo, hi in ((0, 0, n), (L - 300 - n, L - n, L)):
        part = [t[:, a:hi].cpu() for t in (x, dt.clamp(min=-3.5), B, C)]
        ref, mag = (R.scan(part[0], part[1], A, part[2], part[3], skip, None, bias, True, None, None, mag=m) for m in (False, True))
        # as in the operator's own tests, 500 tokens; what came before is e^-90 of it
        R.check(y[:, lo:hi], ref["y"][:, lo - a:], mag["y"][:, lo - a:], 70 * 500 + N + 32, f"y {lo}")
    R.check(h, ref["h_out"], mag["h_out"], 70 * 500 + 16, "h_out")


T, D, N, TAIL = (1 << 20) + 3, 4096, 4, 500


def test_rows_past_the_32_bits():
    """Token arrays of more than 2^32 elements: the last tokens (and the first) of the convolution, the norm, the scan
    and their gradients. A state forgets what lies 300 tokens back (steps of 0.3 at least, |A| of 1 at least)."""
    note(f"{T} tokens of {D} channels, {T * D * 2 >> 20} MiB an array")
    g = torch.Generator(device=device()).manual_seed(8)
    x = torch.empty((1, T, D), dtype=BF16, device=device())
    for i in range(0, T, 1 << 18):
        x[:, i:i + (1 << 18)] = torch.randn(x[:, i:i + (1 << 18)].shape, generator=g, device=device(), dtype=BF16)
    w, bias, nw = rand(gen(1), D, 4, std=0.5), rand(gen(2), D, std=0.5), rand(gen(3), D) + 1
    ends = ((0, 0, TAIL - 300), (T - TAIL, 300, TAIL))       # a slice's first token, and its tokens that are compared

    def cut(t, a, n=TAIL):
        return t[:, a:a + n].cpu()

    y, state = m3.mamba3_conv_fwd(x, up(w), up(bias))
    for a, lo, hi in ends:
        ref, mag = (R.conv(cut(x, a), w, bias, True, None, None, mag=m) for m in (False, True))
        R.check(cut(y, a)[:, lo:hi], ref["y"][:, lo:hi], mag["y"][:, lo:hi], 16, "conv")
    assert torch.equal(state, x[:, T - 3:])
    del y
    gr = m3.mamba3_conv_bwd(x, up(w), up(bias), dy=x)
    for a, lo, hi in ends:
        ref, mag = (R.conv(cut(x, a), w, bias, True, None, None, cut(x, a), None, mag=m) for m in (False, True))
        R.check(cut(gr["dx"], a)[:, lo:hi], ref["dx"][:, lo:hi], mag["dx"][:, lo:hi], 32, "conv dx")
    del gr
    n = m3.mamba3_rmsnorm_fwd(x, up(nw))["y"]
    for a, lo, hi in ends:
        _, v = R.norm(cut(x, a), None, nw, 1e-5)
        R.check(cut(n, a), v, v, LB.norm_count(D), "norm")
    del n
    ds = m3.mamba3_rmsnorm_bwd(x, up(nw), dy=x)["dx"]
    for a, lo, hi in ends:
        ref, mag = (R.norm_bwd(cut(x, a), nw, cut(x, a), None, 1e-5, mag=m)[0] for m in (False, True))
        R.check(cut(ds, a), ref, mag, LB.norm_bwd_count(D), "norm dx")
    del ds
    # one array is x, dt (0.3 .. by its bias), z and dy
    A, skip, db = -1 - rand(gen(4), D, N).abs(), rand(gen(5), D), torch.full((D,), 6.0)
    B, C = (torch.randn((1, T, 1, N), generator=g, device=device(), dtype=BF16) for _ in range(2))
    args = (x, x, up(A), B, C, up(skip))
    kw = dict(z=x, dt_bias=up(db), dt_softplus=True)
    y, h = m3.mamba3_selective_scan_fwd(*args, **kw)
    gr = m3.mamba3_selective_scan_bwd(*args, **kw, dy=x)
    for a, lo, hi in ends:
        p = [cut(t, a) for t in (x, B, C)]
        ref, mag = (R.scan(p[0], p[0], A, p[1], p[2], skip, p[0], db, True, None, None, p[0], None, mag=m) for m in (False, True))
        R.check(cut(y, a)[:, lo:hi], ref["y"][:, lo:hi], mag["y"][:, lo:hi], 70 * TAIL + N + 32, "scan")
        for k in ("dx", "ddt", "dz", "dB", "dC"):
            count = 140 * TAIL + 64 + (D if k in ("dB", "dC") else N)
            R.check(cut(gr[k], a)[:, lo:hi], ref[k][:, lo:hi], mag[k][:, lo:hi], count, k)
        if a:
            R.check(h, ref["h_out"], mag["h_out"], 70 * TAIL + 16, "h_out")


def test_pools_past_the_32_bits():
    """Steps whose slots lie more than 2^32 bytes and 2^31 elements into their pools."""
    b, D, N = 6, 4096, 16
    slots = torch.tensor([3, 33000, 0, 32999, -1, 33001], dtype=torch.int32, device=device())
    g = gen(6)
    x, dt, z = (rand(g, b, D, dtype=BF16) for _ in range(3))
    B, C = (rand(g, b, 1, N, dtype=BF16) for _ in range(2))
    A, start = -torch.exp(rand(g, D, N, std=0.3)), rand(g, b, D, N)
    pool = torch.empty((33001, D, N), device=device())
    note(f"pool of {pool.numel() * 4 >> 20} MiB")
    keep = slots[:4].long()
    pool[keep] = up(start)[:4]
    own = up(start).clone()
    y = m3.mamba3_selective_step(up(x), up(dt), up(A), up(B), up(C), h=pool, z=up(z), dt_softplus=True, slots=slots)
    want = m3.mamba3_selective_step(up(x), up(dt), up(A), up(B), up(C), h=own, z=up(z), dt_softplus=True)
    assert torch.equal(y[:4], want[:4]) and torch.equal(pool[keep], own[:4])
    del pool
    w, start = rand(g, D, 8, std=0.5), rand(g, b, 7, D, dtype=BF16)
    pool, slots = torch.empty((80001, 7, D), dtype=BF16, device=device()), torch.tensor([80000, 5, 79999, 1, 80001, -7],
                                                                                       dtype=torch.int32, device=device())
    keep = slots[:4].long()
    pool[keep] = up(start)[:4]
    own = up(start).clone()
    y, want = m3.mamba3_conv_step(up(x), up(w), conv=pool, slots=slots), m3.mamba3_conv_step(up(x), up(w), conv=own)
    assert torch.equal(y[:4], want[:4]) and torch.equal(pool[keep], own[:4])


@pytest.mark.parametrize("given,means", [([-7, 12, 12, 500], [0, 12, 12, 40]), ([-9, -2, 40], [0, 0, 40]), ([3, 41, 1 << 30], [3, 40, 40]),
                                         ([-(1 << 31), 5, (1 << 31) - 1], [0, 5, 40])])
def test_entries_outside_the_batch(given, means):
    """cu_seqlens' entries are clamped to the tokens that there are."""
    note(f"cu {given}")
    g, L, C = gen(9), 40, 24
    a, kw, dy, dho, _ = scan_inputs((1, L, C, 16, 1, means), BF16, True)
    x, w, cin = up(a["x"]), up(rand(g, C, 4)), up(rand(g, len(means) - 1, 3, C, dtype=BF16))
    res = []
    for cu in (given, means):
        cut = torch.tensor(cu, dtype=torch.int32, device=device())
        o = dict(zip("yc", m3.mamba3_conv_fwd(x, w, conv_in=cin, cu_seqlens=cut)))
        o.update(m3.mamba3_conv_bwd(x, w, dy=up(dy), conv_in=cin, cu_seqlens=cut))
        o["y2"], o["h"] = m3.mamba3_selective_scan_fwd(**dev(a), **dev(kw), cu_seqlens=cut)
        o.update({"s" + k: v for k, v in m3.mamba3_selective_scan_bwd(**dev(a), **dev(kw), dy=up(dy), dh_out=up(dho), cu_seqlens=cut).items()})
        res.append(o)
    lo, hi = means[0], means[-1]
    for k, t in res[0].items():
        other = res[1][k]
        if t.dim() > 1 and t.shape[:2] == (1, L):
            t, other = t[:, lo:hi], other[:, lo:hi]
        assert torch.equal(t, other), k
