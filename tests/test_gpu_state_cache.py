"""The cache of states on the GPU: every byte, scale and value read back equals its 64-bit form's
(tests/gated_ref.py): the roundings are all defined."""
import pytest
import torch

import state_space_sequence_mamba3_amd as m3
from tests import gated_ref as R
from tests.gpu_util import device, note

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
KINDS = ["e4m3", "int8", "int4"]


def up(t):
    return t.to(device()) if t is not None else None


def same(a, b):
    """Bit for bit, NaNs as NaNs."""
    a, b = a.cpu(), b.cpu()
    assert a.dtype == b.dtype and a.shape == b.shape
    if a.dtype == torch.float8_e4m3fn:
        a, b = a.float(), b.float()
    return torch.equal(a, b) or (a.is_floating_point() and torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0)))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("block", [32, 64, 128, 256])
@pytest.mark.parametrize("values", [1, 7, 8, 31, 33, 64, 257, 2048, 2049, 5000])
def test_round(values, block, kind, dtype):
    note(f"cache {kind} block {block} values {values} {dtype}")
    g = torch.Generator().manual_seed(values + block)
    h = (torch.randn(5, values, generator=g) * torch.exp(2 * torch.randn(5, values, generator=g))).to(dtype)
    want, scale = R.store(h, kind, block)
    q, s = m3.mamba3_state_store(up(h), kind=kind, block=block)
    assert same(s, scale) and same(q, want)
    back = torch.zeros_like(up(h))
    out = m3.mamba3_state_load(q, s, h=back, kind=kind, block=block)
    assert out is back and same(back, R.load(want, scale, kind, block, values, dtype))


@pytest.mark.parametrize("kind", KINDS)
def test_quotients(kind):
    """A million values over all magnitudes, blocks of subnormal, tiny and huge ones: the quotient is the rounded
    one everywhere."""
    g = torch.Generator().manual_seed(3)
    h = torch.randn(64, 16384, generator=g).view(64, 512, 32)
    h = (h * torch.exp2(torch.randint(-148, 126, (64, 512, 1), generator=g).double())).float().view(64, -1)
    want, scale = R.store(h, kind, 32)
    q, s = m3.mamba3_state_store(up(h), kind=kind, block=32)
    assert same(s, scale) and same(q, want)
    assert same(m3.mamba3_state_load(q, s, h=torch.empty_like(up(h)), kind=kind, block=32), R.load(want, scale, kind, 32, 16384, F32))


@pytest.mark.parametrize("kind", KINDS)
def test_ties(kind):
    """Values halfway between two of the kind, with a scale that is a power of two: ties go to even."""
    top = R.TOP[kind]
    v = torch.arange(0, 2 * top + 1) / 2
    v = torch.cat([v, -v])
    n = -(-v.numel() // 31)
    h = torch.full((1, n * 32), top).view(n, 32)
    h[:, 1:] = torch.cat([v, torch.zeros(n * 31 - v.numel())]).view(n, 31)
    h = h.view(1, -1) * 0.5
    want, scale = R.store(h, kind, 32)
    q, s = m3.mamba3_state_store(up(h), kind=kind, block=32)
    assert bool((s == 0.5).all()) and same(q, want)


@pytest.mark.parametrize("kind", KINDS)
def test_not_finite_and_zero(kind):
    h = torch.randn(3, 200, generator=torch.Generator().manual_seed(1))
    h[0, 3], h[0, 70], h[1, 199], h[2, 64:128] = float("inf"), float("nan"), float("-inf"), 0.0
    want, scale = R.store(h, kind, 64)
    q, s = m3.mamba3_state_store(up(h), kind=kind, block=64)
    assert same(s, scale) and float(s[2, 1]) == 2.0 ** -126
    back = m3.mamba3_state_load(q, s, h=torch.empty_like(up(h)), kind=kind, block=64).cpu()
    assert bool(back[0, :128].isnan().all()) and bool(back[0, 128:].isfinite().all())
    assert bool(back[1, 192:].isnan().all()) and bool(back[1, :192].isfinite().all())
    assert bool((back[2, 64:128] == 0).all()) and bool(back[2].isfinite().all())


@pytest.mark.parametrize("kind", ["int8", "int4", "e4m3"])
@pytest.mark.parametrize("values", [300, 301])
def test_every_byte(kind, values):
    """Loading takes any bytes."""
    g = torch.Generator().manual_seed(4)
    n = (values + 1) // 2 if kind == "int4" else values
    raw = torch.arange(4 * n).remainder(256).to(torch.uint8).view(4, n)
    q = raw if kind == "int4" else raw.view(torch.int8 if kind == "int8" else torch.float8_e4m3fn)
    s = torch.rand(4, -(-values // 128), generator=g)
    for dtype in (F32, BF16):
        got = m3.mamba3_state_load(up(q), up(s), h=torch.empty(4, values, dtype=dtype, device=device()), kind=kind, block=128)
        assert same(got, R.load(q, s, kind, 128, values, dtype))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", [(4, 8, 6), (37,)])
def test_slots_and_entries(kind, shape):
    """States picked by slots into entries and back into other slots; rows out of range are skipped, and what
    is not named stays. The same entry may be read into several slots."""
    g = torch.Generator().manual_seed(6)
    h = torch.randn(9, *shape, generator=g)
    values = h[0].numel()
    want, scale = R.store(h.view(9, -1), kind, 32)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=device())   # noqa: E731
    q = torch.full((6, want.shape[1]), 1.0).to(want.dtype)
    s = torch.full((6, scale.shape[1]), 3.0)
    qd, sd = up(q), up(s)
    m3.mamba3_state_store(up(h), kind=kind, block=32, slots=i32(8, 0, -1, 9, 3, 5), entries=i32(1, 5, 0, 0, 6, 2), q=qd, scale=sd)
    for slot, e in ((8, 1), (0, 5), (5, 2)):
        q[e], s[e] = want[slot], scale[slot]
    assert same(qd, q) and same(sd, s)
    pool = torch.full((4, *shape), 2.0)
    on = up(pool)
    m3.mamba3_state_load(qd, sd, h=on, kind=kind, block=32, slots=i32(3, 1, 0, 4, -2), entries=i32(5, 5, 2, 1, 1))
    for slot, e in ((3, 5), (1, 5), (0, 2)):
        pool[slot] = R.load(q[e:e + 1], s[e:e + 1], kind, 32, values, F32).view(shape)
    assert torch.equal(on.cpu(), pool)


def test_guards():
    """Nothing is written outside an odd state's place."""
    for kind in KINDS:
        n = 17 if kind == "int4" else 33
        h = torch.randn(3, 33, generator=torch.Generator().manual_seed(2))
        want, scale = R.store(h, kind, 32)
        raw = torch.full((3 * n + 2,), 77, dtype=torch.uint8, device=device())
        q = raw[1:-1].view(want.dtype).view(3, n)
        m3.mamba3_state_store(up(h), kind=kind, block=32, q=q, scale=torch.empty(3, 2, device=device()))
        assert same(q, want) and int(raw[0]) == 77 and int(raw[-1]) == 77
        room = torch.full((3 * 33 + 2,), 7.0, device=device())
        m3.mamba3_state_load(q, up(scale), h=room[1:-1].view(3, 33), kind=kind, block=32)
        assert float(room[0]) == 7 and float(room[-1]) == 7
