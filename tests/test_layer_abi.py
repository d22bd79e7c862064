"""The layer operators' C ABI and binding on the CPU: struct layouts, every refusal of the host
validation, and the binding's own checks. No compute call is made here."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import state_space_sequence_mamba3_amd as m3
from tests import layer_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = {"mamba3_conv_args": m3.ConvArgs, "mamba3_conv_bwd_args": m3.ConvBwdArgs,
           "mamba3_conv_step_args": m3.ConvStepArgs, "mamba3_selective_scan_args": m3.SelectiveScanArgs,
           "mamba3_selective_scan_bwd_args": m3.SelectiveScanBwdArgs,
           "mamba3_selective_step_args": m3.SelectiveStepArgs, "mamba3_rmsnorm_args": m3.RmsnormArgs,
           "mamba3_rmsnorm_bwd_args": m3.RmsnormBwdArgs}
OK, EINVAL, EUNSUPPORTED, EALIGN, EWORKSPACE = (m3.MAMBA3_OK, m3.MAMBA3_EINVAL, m3.MAMBA3_EUNSUPPORTED,
                                                m3.MAMBA3_EALIGN, m3.MAMBA3_EWORKSPACE)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(m3.LIB_PATH):
        from state_space_sequence_mamba3_amd import build
        build.build()
    return m3.lib()


def test_struct_layouts(tmp_path):
    """Every field of the binding's structs lies where the C compiler puts it."""
    lines = []
    for name, cls in STRUCTS.items():
        lines.append(f'printf("{name} . %zu\\n", sizeof({name}));')
        lines += [f'printf("{name} {f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include "mamba3.h"\nint main(void) {\n' + "\n".join(lines) + "\nreturn 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines():
        name, field, n = line.split()
        cls = STRUCTS[name]
        assert int(n) == (ctypes.sizeof(cls) if field == "." else getattr(cls, field).offset), line
    header = open(os.path.join(ROOT, "include", "mamba3.h")).read()
    for name, cls in STRUCTS.items():       # no field of the header is missing here
        body = re.sub(r"/\*.*?\*/", "", header[:header.index("} " + name + ";")].rsplit("typedef struct {", 1)[1], flags=re.S)
        assert sum(d.count(",") + 1 for d in body.split(";") if d.strip()) == len(cls._fields_), name


def fake(i):
    return 0x7E0000000000 + i * 0x100000000


def conv(**o):
    return build(m3.ConvArgs, dict(batch=2, seqlen=10, dim=16, width=4, dtype=m3.MAMBA3_BF16, silu=1, x=fake(1),
                                   weight=fake(2), bias=fake(3), conv_in=fake(4), y=fake(5), conv_out=fake(6)), o)


def conv_bwd(**o):
    f = {k[4:]: o.pop(k) for k in list(o) if k.startswith("fwd_")}
    return build(m3.ConvBwdArgs, dict(fwd=conv(**f), dy=fake(7), dconv_out=fake(8), dx=fake(9), dweight=fake(10),
                                      dbias=fake(11), dconv_in=fake(12), workspace=fake(13), workspace_bytes=1 << 30), o)


def conv_step(**o):
    return build(m3.ConvStepArgs, dict(batch=3, dim=16, width=4, dtype=m3.MAMBA3_F32, silu=0, x=fake(1),
                                       weight=fake(2), bias=fake(3), conv=fake(4), y=fake(5)), o)


def scan(**o):
    return build(m3.SelectiveScanArgs, dict(batch=2, seqlen=10, dim=16, dstate=16, ngroups=2, dtype=m3.MAMBA3_BF16,
                                            dt_softplus=1, x=fake(1), dt=fake(2), B=fake(3), C=fake(4), z=fake(5),
                                            A=fake(6), D=fake(7), dt_bias=fake(8), h_in=fake(9), y=fake(10),
                                            h_out=fake(11), workspace=fake(30), workspace_bytes=1 << 30), o)


def scan_bwd(**o):
    f = {k[4:]: o.pop(k) for k in list(o) if k.startswith("fwd_")}
    return build(m3.SelectiveScanBwdArgs, dict(fwd=scan(**f), dy=fake(12), dh_out=fake(13), dx=fake(14), ddt=fake(15),
                                               dB=fake(16), dC=fake(17), dz=fake(18), dA=fake(19), dD=fake(20),
                                               ddt_bias=fake(21), dh_in=fake(22), workspace=fake(31),
                                               workspace_bytes=1 << 30), o)


def step(**o):
    return build(m3.SelectiveStepArgs, dict(batch=3, dim=16, dstate=16, ngroups=1, dtype=m3.MAMBA3_F32, x=fake(1),
                                            dt=fake(2), B=fake(3), C=fake(4), z=fake(5), A=fake(6), D=fake(7),
                                            dt_bias=fake(8), h=fake(9), y=fake(10)), o)


def norm(**o):
    return build(m3.RmsnormArgs, dict(rows=5, dim=300, dtype=m3.MAMBA3_BF16, residual_dtype=m3.MAMBA3_F32,
                                      qtype=m3.MAMBA3_E4M3, qblock=128, eps=1e-5, x=fake(1), residual=fake(2),
                                      weight=fake(3), residual_out=fake(4), y=fake(5), q=fake(6), qscale=fake(7)), o)


def norm_bwd(**o):
    return build(m3.RmsnormBwdArgs, dict(rows=5, dim=300, dtype=m3.MAMBA3_BF16, residual_dtype=m3.MAMBA3_F32, eps=1e-5,
                                         s=fake(1), dy=fake(2), dresidual_out=fake(3), weight=fake(4), dx=fake(5),
                                         dresidual=fake(6), dweight=fake(7), workspace=fake(8),
                                         workspace_bytes=1 << 30), o)


def build(cls, fields, over):
    a = cls()
    for k, v in {**fields, **over}.items():
        setattr(a, k, v)
    return a


NAMES = {m3.ConvArgs: "conv", m3.ConvBwdArgs: "conv_bwd", m3.ConvStepArgs: "conv_step",
         m3.SelectiveScanArgs: "selective_scan", m3.SelectiveScanBwdArgs: "selective_scan_bwd",
         m3.SelectiveStepArgs: "selective_step", m3.RmsnormArgs: "rmsnorm", m3.RmsnormBwdArgs: "rmsnorm_bwd"}

CASES = [
    # accepted
    (conv, {}, OK), (conv, dict(bias=None, conv_in=None, conv_out=None), OK), (conv, dict(seqlen=0, x=None, y=None), OK),
    (conv, dict(batch=0), OK), (conv, dict(x=fake(1) + 2, x_row=33), OK),
    (conv, dict(batch=1, cu_seqlens=fake(20), nseq=3), OK), (conv_bwd, {}, OK),
    (conv_bwd, dict(dconv_in=None, dbias=None, dconv_out=None), OK), (conv_step, {}, OK), (conv_step, dict(batch=0), OK),
    (conv_step, dict(slots=fake(20), nslots=9), OK), (scan, {}, OK), (scan, dict(h_out=fake(9)), OK),
    (scan, dict(z=None, D=None, dt_bias=None, h_in=None, h_out=None), OK), (scan, dict(dstate=128), OK),
    (scan, dict(dstate=1, x_row=40, B_row=50), OK), (scan, dict(batch=0), OK), (scan_bwd, dict(fwd_batch=0), OK),
    (scan, dict(seqlen=0), OK), (scan_bwd, dict(fwd_seqlen=0), OK), (conv_bwd, dict(fwd_batch=0), OK),
    (norm_bwd, dict(rows=0), OK), (scan, dict(batch=1, seqlen=1 << 20, dim=2), OK), (norm, dict(rows=0, y=None, q=None, qscale=None), OK), (scan_bwd, {}, OK), (scan_bwd, dict(dz=None, dD=None, dh_in=None), OK),
    (step, {}, OK), (step, dict(batch=0), OK), (norm, {}, OK), (norm, dict(q=None, qscale=None), OK),
    (norm, dict(y=None), OK), (norm, dict(residual_out=fake(2)), OK), (norm, dict(rows=0), OK), (norm, dict(qblock=0), OK),
    (norm, dict(qblock=300), OK), (norm, dict(qtype=m3.MAMBA3_INT8, qblock=32), OK), (norm_bwd, {}, OK),
    (norm_bwd, dict(dresidual=fake(3)), OK), (norm_bwd, dict(dweight=None, workspace=None, workspace_bytes=0), OK),
    # sizes and flags
    (conv, dict(dtype=2), EINVAL), (conv, dict(silu=2), EINVAL), (conv, dict(dim=0), EINVAL), (conv, dict(batch=-1), EINVAL),
    (conv, dict(seqlen=-1), EINVAL), (conv, dict(width=0), EINVAL), (conv, dict(width=1), EUNSUPPORTED),
    (conv, dict(width=9), EUNSUPPORTED), (conv, dict(x_row=15), EINVAL), (conv, dict(x_row=-16), EINVAL),
    (conv, dict(x_row=1 << 31), EINVAL), (conv, dict(cu_seqlens=fake(20), nseq=3), EINVAL),
    (conv, dict(batch=1, cu_seqlens=fake(20), nseq=0), EINVAL), (conv, dict(batch=1 << 20, seqlen=1 << 12), EINVAL),
    (conv_bwd, dict(dy_row=3), EINVAL), (conv_bwd, dict(fwd_conv_in=None), EINVAL), (conv_step, dict(width=1), EUNSUPPORTED),
    (conv_step, dict(slots=fake(20), nslots=-1), EINVAL), (conv_step, dict(dim=-4), EINVAL),
    (scan, dict(ngroups=3), EINVAL), (scan, dict(dstate=0), EINVAL), (scan, dict(dstate=129), EUNSUPPORTED),
    (scan, dict(dt_softplus=-1), EINVAL), (scan, dict(B_row=31), EINVAL), (scan, dict(z_row=1), EINVAL),
    (scan, dict(batch=1 << 20, seqlen=1 << 12), EINVAL), (scan_bwd, dict(fwd_z=None), EINVAL),
    (scan_bwd, dict(fwd_dstate=200), EUNSUPPORTED), (scan_bwd, dict(dy_row=2), EINVAL), (step, dict(ngroups=5), EINVAL),
    (step, dict(dstate=129), EUNSUPPORTED), (step, dict(C_row=7), EINVAL),
    (norm, dict(eps=-1.0), EINVAL), (norm, dict(eps=float("nan")), EINVAL), (norm, dict(eps=float("inf")), EINVAL),
    (norm, dict(rows=-1), EINVAL), (norm, dict(dim=0), EINVAL), (norm, dict(qblock=100), EUNSUPPORTED),
    (norm, dict(qblock=-1), EINVAL), (norm, dict(qtype=2), EINVAL), (norm, dict(q=None), EINVAL),
    (norm, dict(y=None, q=None, qscale=None), EINVAL), (norm, dict(dtype=m3.MAMBA3_F32, residual_dtype=m3.MAMBA3_BF16),
                                                        EUNSUPPORTED), (norm_bwd, dict(dx=None, dresidual=None), EINVAL),
    # required pointers
    *[(f, {k: None}, EINVAL) for f, ks in ((conv, ("x", "weight", "y")), (conv_bwd, ("dy", "dx", "dweight")),
                                           (conv_step, ("x", "weight", "y", "conv")), (scan, ("x", "dt", "B", "C", "A", "y")),
                                           (scan_bwd, ("dy", "dx", "ddt", "dB", "dC", "dA")),
                                           (step, ("x", "dt", "B", "C", "A", "h", "y")), (norm, ("x",)),
                                           (norm_bwd, ("s", "dy"))) for k in ks],
    # alignment
    (conv, dict(x=fake(1) + 1), EALIGN), (conv, dict(weight=fake(2) + 2), EALIGN), (conv_bwd, dict(workspace=fake(13) + 16),
                                                                                   EALIGN),
    (scan, dict(A=fake(6) + 4), EALIGN), (scan, dict(h_in=fake(9) + 8), EALIGN), (step, dict(h=fake(9) + 4), EALIGN),
    (scan_bwd, dict(dh_out=fake(13) + 4), EALIGN), (norm, dict(residual=fake(2) + 2), EALIGN),
    (conv, dict(batch=1, cu_seqlens=fake(20) + 2, nseq=1), EALIGN),
    # overlaps
    (conv, dict(y=fake(1)), EINVAL), (conv, dict(conv_out=fake(4)), EINVAL), (conv, dict(conv_out=fake(5) + 32), EINVAL),
    (conv_bwd, dict(dx=fake(7)), EINVAL), (conv_bwd, dict(dweight=fake(11)), EINVAL), (conv_step, dict(y=fake(4)), EINVAL),
    (scan, dict(y=fake(5)), EINVAL), (scan, dict(h_out=fake(9) + 16), EINVAL), (scan, dict(y=fake(11)), EINVAL),
    (scan, dict(workspace=fake(1)), EINVAL), (scan_bwd, dict(dB=fake(17)), EINVAL), (scan_bwd, dict(dh_in=fake(13)), EINVAL),
    (scan_bwd, dict(workspace=fake(14)), EINVAL), (step, dict(y=fake(9)), EINVAL), (norm, dict(y=fake(1)), EINVAL),
    (norm, dict(residual_out=fake(2) + 4), EINVAL), (norm_bwd, dict(dx=fake(2)), EINVAL),
    (conv, dict(x_row=100, y=fake(1) + 2 * 100 * 15), EINVAL),      # inside the last rows of a strided x
    # workspaces
    (conv_bwd, dict(workspace=None, workspace_bytes=0), EWORKSPACE), (conv_bwd, dict(workspace_bytes=16), EWORKSPACE),
    (scan_bwd, dict(workspace_bytes=64), EWORKSPACE), (norm_bwd, dict(workspace=None), EWORKSPACE),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_validation(lib, i):
    make, over, want = CASES[i]
    a = make(**over)
    name = NAMES[type(a)]
    assert getattr(lib, f"mamba3_{name}_validate")(ctypes.byref(a)) == want, (name, over)
    if want != OK:      # the entry point refuses the same before any HIP call
        run = f"mamba3_{name}" + ("_fwd" if name in ("conv", "selective_scan", "rmsnorm") else "")
        assert getattr(lib, run)(ctypes.byref(a), None) == want


def test_null_arguments(lib):
    for n in m3.LAYER_EXPORTS:
        f = getattr(lib, n)
        if n.endswith("_validate"):
            assert f(None) == EINVAL
        elif n.endswith("_size"):
            assert f(None) == 0
        else:
            assert f(None, None) == EINVAL


def test_workspace_sizes(lib):
    size = lambda a: getattr(lib, f"mamba3_{NAMES[type(a)]}_workspace_size")(ctypes.byref(a))   # noqa: E731
    assert size(conv_bwd()) > 0 and size(conv_bwd(fwd_width=9)) == 0
    assert size(scan_bwd()) > size(scan_bwd(fwd_seqlen=1)) > 0 and size(scan_bwd(fwd_dstate=129)) == 0
    assert size(norm_bwd()) > 0 and size(norm_bwd(dweight=None)) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(1, 4, 8)
    w = torch.zeros(8, 4)
    with pytest.raises(ValueError, match="device memory"):
        m3.mamba3_conv_fwd(x, w)
    with pytest.raises(ValueError, match="dimensions"):
        m3.mamba3_conv_fwd(x[0], w)
    with pytest.raises(ValueError, match="device memory"):
        m3.mamba3_conv_step(x[0], w, conv=torch.zeros(4, 3, 8))
    with pytest.raises(ValueError, match="device memory"):
        m3.mamba3_selective_step(x[0], x[0], torch.zeros(8, 2), torch.zeros(4, 1, 2), torch.zeros(4, 1, 2),
                                 h=torch.zeros(4, 8, 2))
    with pytest.raises(ValueError, match="device memory"):
        m3.mamba3_rmsnorm_fwd(x)
    with pytest.raises(ValueError, match="dy must have shape"):
        m3.mamba3_rmsnorm_bwd(x, dy=x[0])


def test_token_rows():
    """Which views count as token rows, and their distance."""
    from state_space_sequence_mamba3_amd.layer import _rows
    cpu = -1

    def row(t, lead):
        return _rows(t, t.shape, lead, t.dtype, cpu, "t")[1]

    t = torch.zeros(3, 5, 24)
    assert row(t, 2) == 0 and row(t[:, :, 4:12], 2) == 24 and row(t[:, 0], 1) == 120 and row(t[:1, :, :8], 2) == 24
    assert row(t[:, :1, :8], 2) == 120 and row(t[1:2, 2:3, :7], 2) == 0
    assert row(t[:, :, 2:18].unflatten(2, (2, 8)), 2) == 24
    for bad, lead in ((t[:, ::2, :8], 2), (t[:, :3], 2), (t.transpose(0, 1), 2), (t[:, :, ::2], 2),
                      (t[:, :, :1].expand(3, 5, 8), 2), (t[:, :1].expand(3, 4, 24), 2),
                      (t[:, :, :16].unflatten(2, (2, 8)).transpose(2, 3), 2)):
        with pytest.raises(ValueError):
            row(bad, lead)


def test_planted_mistakes_are_seen():
    """The references' comparison fails for an error of a thousandth in 32 bits and of one step in bf16."""
    g = torch.Generator().manual_seed(1)
    x, w = torch.randn(1, 9, 8, generator=g), torch.randn(8, 4, generator=g)
    ref, mag = R.conv(x, w, None, True, None, None), R.conv(x, w, None, True, None, None, mag=True)
    R.check(ref["y"].float(), ref["y"], mag["y"], 16, "y")
    R.check(ref["y"].bfloat16(), ref["y"], mag["y"], 16, "y")
    for wrong in (ref["y"].float() * 1.001, (ref["y"] * 1.01).bfloat16(), ref["y"].float().roll(1, 1)):
        with pytest.raises(AssertionError):
            R.check(wrong, ref["y"], mag["y"], 16, "y")
