"""States read back from the cache to bf16: q scale is rounded once, from the exact product."""
import numpy as np
import pytest
import torch

import state_space_sequence_mamba3_amd as m3
from tests.gpu_util import device, note

pytestmark = pytest.mark.gpu


def rounded(v):
    """Doubles to the nearest bf16, ties to even (by their significands, not by way of fp32)."""
    v = np.asarray(v, np.float64)
    _, e = np.frexp(v)
    unit = np.maximum(e - 8, -133)                      # a bf16's last place; the subnormals'
    r = np.ldexp(np.rint(np.ldexp(v, -unit)), unit)     # (a quotient by a power of two is exact, rint takes ties to even)
    return np.where(np.abs(r) >= 2.0 ** 128, np.copysign(np.inf, r), r)


def near_ties(g, values):
    """(place in `values`, scale): products that lie next to the middle of two bf16 values, on either side, so near
    that fp32 holds the middle; and ordinary ones, down to subnormal products."""
    out = [(int((values == 127).nonzero()[0, 0]), 4276869.0)] if bool((values == 127).any()) else []
    odd = [k for k, v in enumerate(values.tolist()) if v and np.isfinite(v) and np.frexp(v)[0] not in (0.5, -0.5)]
    while len(out) < 3000:
        k = odd[int(torch.randint(len(odd), (1,), generator=g))]
        mid = (int(torch.randint(128, 256, (1,), generator=g)) + 0.5) * 2.0 ** int(torch.randint(-120, 100, (1,), generator=g))
        s = np.float32(abs(mid / float(values[k])))
        for c in (s, np.nextafter(s, np.float32(np.inf)), np.nextafter(s, np.float32(0))):
            p = float(c) * abs(float(values[k]))
            if p != mid and np.float64(np.float32(p)) == mid:
                out.append((k, float(c)))
                break
        else:
            if len(out) % 7 == 0:
                out.append((k, float(torch.exp2(torch.rand((), generator=g) * 250 - 126))))
    return out


@pytest.mark.parametrize("kind", ["e4m3", "int8", "int4"])
def test_one_rounding(kind):
    note(f"cache read back to bf16 {kind}")
    g = torch.Generator().manual_seed(5)
    raw = torch.arange(256, dtype=torch.uint8)
    if kind == "e4m3":
        values = raw.view(torch.float8_e4m3fn).double()
    elif kind == "int8":
        values = raw.view(torch.int8).double()
    else:
        values = torch.arange(16).double()
        values = values - 16 * (values >= 8)
    pairs = near_ties(g, values)
    n, block = len(pairs), 32
    # entries of one block: the pair's value, and others
    place = torch.randint(len(values), (n, block), generator=g)
    place[:, 0] = torch.tensor([k for k, _ in pairs])
    place[:, 17] = place[:, 0]
    scale = torch.tensor([s for _, s in pairs]).float().view(n, 1)
    v = values[place]
    want = rounded((v * scale.double()).nan_to_num(7.0).numpy())
    by_fp32 = (v.float() * scale).bfloat16().double().nan_to_num(7.0).numpy()
    assert (want != by_fp32).sum() > 1000                # (rounded twice, these differ)
    q = (place[:, 0::2] | place[:, 1::2] << 4).to(torch.uint8) if kind == "int4" else raw[place].view(
        torch.int8 if kind == "int8" else torch.float8_e4m3fn)
    got = m3.mamba3_state_load(q.to(device()), scale.to(device()), h=torch.empty(n, block, dtype=torch.bfloat16, device=device()),
                               kind=kind, block=block).cpu().double()
    assert torch.equal(got.isnan(), v.isnan())
    assert np.array_equal(got.nan_to_num(7.0, posinf=float("inf"), neginf=float("-inf")).numpy(), want)


@pytest.mark.parametrize("kind", ["e4m3", "int8", "int4"])
def test_scales_of_any_bits(kind):
    """An infinite scale reads back as infinities and, times zero, NaN; a NaN one as NaN; a product past the range as
    an infinity."""
    one = {"e4m3": 0x38, "int8": 1, "int4": 0x11}[kind]
    n = 16 if kind == "int4" else 32
    ty = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8, "int4": torch.uint8}[kind]
    q = torch.full((4, n), one, dtype=torch.uint8)
    q[:, :8] = 0
    s = torch.tensor([[float("inf")], [float("nan")], [3.4e38], [float("-inf")]])
    got = m3.mamba3_state_load(q.view(ty).to(device()), s.to(device()), h=torch.empty(4, 32, dtype=torch.bfloat16, device=device()),
                               kind=kind, block=32).cpu().float()
    z = 16 if kind == "int4" else 8
    assert bool(got[0, :z].isnan().all()) and bool((got[0, z:] == float("inf")).all())
    assert bool(got[1].isnan().all())
    assert bool((got[2, :z] == 0).all()) and bool((got[2, z:] == float("inf")).all())      # (above the middle of bf16's last and infinity)
    assert bool(got[3, :z].isnan().all()) and bool((got[3, z:] == float("-inf")).all())
