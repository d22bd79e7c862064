"""The gated layer's operators' C ABI and binding on the CPU: struct layouts, every refusal of the host
validation, the documented sizes, and the binding's own checks. No compute call is made here."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import state_space_sequence_mamba3_amd as m3
from tests.test_layer_abi import EALIGN, EINVAL, EUNSUPPORTED, EWORKSPACE, OK, ROOT, build, fake
from tests.test_layer_abi import lib  # noqa: F401  (a fixture)

STRUCTS = {"mamba3_gated_scan_args": m3.GatedScanArgs, "mamba3_gated_scan_bwd_args": m3.GatedScanBwdArgs,
           "mamba3_gated_step_args": m3.GatedStepArgs, "mamba3_groupnorm_args": m3.GroupnormArgs,
           "mamba3_groupnorm_bwd_args": m3.GroupnormBwdArgs, "mamba3_state_cache_args": m3.StateCacheArgs}
NAMES = {cls: name[len("mamba3_"):-len("_args")] for name, cls in STRUCTS.items()}
F32, BF16 = m3.MAMBA3_F32, m3.MAMBA3_BF16


def test_struct_layouts(tmp_path):
    """Every field of the binding's structs lies where the C compiler puts it."""
    lines = []
    for name, cls in STRUCTS.items():
        lines.append(f'printf("{name} . %zu\\n", sizeof({name}));')
        lines += [f'printf("{name} {f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "mamba3.h"\n#if MAMBA3_LAYER_OPERATORS < 2\n#error missing\n'
                   '#endif\nint main(void) {\n' + "\n".join(lines) + "\nreturn 0; }\n")
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


def scan(**o):
    return build(m3.GatedScanArgs, dict(batch=2, seqlen=10, dim=16, dtype=BF16, form=m3.MAMBA3_GATE_DECAY, rate=8.0, x=fake(1),
                                        gate=fake(2), i=fake(3), z=fake(4), weight=fake(5), h_in=fake(6), y=fake(7),
                                        h_out=fake(8), workspace=fake(30), workspace_bytes=1 << 30), o)


def scan_bwd(**o):
    f = {k[4:]: o.pop(k) for k in list(o) if k.startswith("fwd_")}
    return build(m3.GatedScanBwdArgs, dict(fwd=scan(**f), dy=fake(9), dh_out=fake(10), dx=fake(11), dgate=fake(12), di=fake(13),
                                           dz=fake(14), dweight=fake(15), dh_in=fake(16), workspace=fake(31),
                                           workspace_bytes=1 << 30), o)


def step(**o):
    return build(m3.GatedStepArgs, dict(batch=3, dim=16, dtype=F32, form=m3.MAMBA3_GATE_FORGET, x=fake(1), gate=fake(2),
                                        i=fake(3), z=fake(4), weight=fake(5), h=fake(6), y=fake(7)), o)


def norm(**o):
    return build(m3.GroupnormArgs, dict(rows=5, dim=300, groups=3, dtype=BF16, act=m3.MAMBA3_GN_GATE, center=1, eps=1e-5, x=fake(1),
                                        z=fake(2), weight=fake(3), bias=fake(4), y=fake(5)), o)


def norm_bwd(**o):
    f = {k[4:]: o.pop(k) for k in list(o) if k.startswith("fwd_")}
    return build(m3.GroupnormBwdArgs, dict(fwd=norm(**f), dy=fake(6), dx=fake(7), dz=fake(8), dweight=fake(9), dbias=fake(10),
                                           workspace=fake(11), workspace_bytes=1 << 30), o)


def cache(**o):
    return build(m3.StateCacheArgs, dict(n=3, values=100, dtype=F32, kind=m3.MAMBA3_CACHE_INT8, block=64, nslots=9, nentries=7,
                                         slots=fake(1), entries=fake(2), h=fake(3), q=fake(4), scale=fake(5)), o)


CASES = [
    # accepted
    (scan, {}, OK), (scan, dict(i=None, z=None, h_in=None, h_out=None), OK), (scan, dict(h_out=fake(6)), OK),
    (scan, dict(form=m3.MAMBA3_GATE_FORGET, weight=None, rate=float("nan")), OK), (scan, dict(batch=0), OK),
    (scan, dict(seqlen=0, x=None, gate=None, y=None), OK), (scan, dict(x=fake(1) + 2, x_row=17, gate_row=33), OK),
    (scan, dict(batch=1, cu_seqlens=fake(20), nseq=3), OK), (scan, dict(rate=0.0), OK), (scan_bwd, {}, OK),
    (scan_bwd, dict(di=None, dz=None, dweight=None, dh_in=None, dh_out=None), OK), (scan_bwd, dict(fwd_batch=0), OK),
    (scan_bwd, dict(fwd_seqlen=0), OK), (scan_bwd, dict(fwd_h_in=None), OK), (step, {}, OK), (step, dict(batch=0), OK),
    (step, dict(weight=None, i=None, z=None), OK), (step, dict(slots=fake(20), nslots=9), OK), (norm, {}, OK),
    (norm, dict(weight=None, bias=None), OK), (norm, dict(act=m3.MAMBA3_GN_NONE, z=None), OK), (norm, dict(rows=0), OK),
    (norm, dict(rows=0, x=None, z=None, y=None), OK), (norm, dict(dim=8192, groups=1), OK), (norm_bwd, {}, OK),
    (norm_bwd, dict(dz=None), OK), (norm_bwd, dict(dweight=None, dbias=None, workspace=None, workspace_bytes=0), OK),
    (cache, {}, OK), (cache, dict(n=0), OK), (cache, dict(slots=None, entries=None), OK), (cache, dict(kind=m3.MAMBA3_CACHE_INT4, block=256), OK),
    (cache, dict(nslots=0), OK), (cache, dict(nentries=0), OK),
    # sizes and flags
    (scan, dict(dtype=2), EINVAL), (scan, dict(form=2), EINVAL), (scan, dict(form=-1), EINVAL), (scan, dict(dim=0), EINVAL),
    (scan, dict(batch=-1), EINVAL), (scan, dict(seqlen=-1), EINVAL), (scan, dict(x_row=15), EINVAL), (scan, dict(gate_row=-16), EINVAL),
    (scan, dict(i_row=3), EINVAL), (scan, dict(z_row=1 << 31), EINVAL), (scan, dict(rate=-1.0), EINVAL),
    (scan, dict(rate=float("inf")), EINVAL), (scan, dict(rate=float("nan")), EINVAL), (scan, dict(cu_seqlens=fake(20), nseq=3), EINVAL),
    (scan, dict(batch=1, cu_seqlens=fake(20), nseq=0), EINVAL), (scan, dict(batch=1 << 20, seqlen=1 << 12), EINVAL),
    (scan_bwd, dict(dy_row=2), EINVAL), (scan_bwd, dict(fwd_i=None), EINVAL), (scan_bwd, dict(fwd_z=None), EINVAL),
    (scan_bwd, dict(fwd_form=m3.MAMBA3_GATE_FORGET, fwd_weight=None), EINVAL), (step, dict(slots=fake(20), nslots=-1), EINVAL),
    (step, dict(dim=0), EINVAL), (step, dict(form=m3.MAMBA3_GATE_DECAY, rate=-2.0), EINVAL), (step, dict(gate_row=7), EINVAL),
    (norm, dict(groups=7), EINVAL), (norm, dict(groups=0), EINVAL), (norm, dict(act=4), EINVAL), (norm, dict(act=-1), EINVAL),
    (norm, dict(center=2), EINVAL), (norm, dict(eps=-1.0), EINVAL), (norm, dict(eps=float("nan")), EINVAL), (norm, dict(rows=-1), EINVAL),
    (norm, dict(act=m3.MAMBA3_GN_SILU), EINVAL), (norm, dict(dim=8193, groups=1), EUNSUPPORTED), (norm, dict(x_row=200), EINVAL),
    (norm, dict(rows=1 << 31, groups=4, dim=400), EINVAL),
    (norm_bwd, dict(dy_row=7), EINVAL), (norm_bwd, dict(fwd_act=m3.MAMBA3_GN_NONE, fwd_z=None), EINVAL),
    (norm_bwd, dict(fwd_weight=None), EINVAL), (norm_bwd, dict(fwd_bias=None), EINVAL),
    (cache, dict(kind=3), EINVAL), (cache, dict(kind=-1), EINVAL), (cache, dict(block=16), EUNSUPPORTED), (cache, dict(block=0), EUNSUPPORTED),
    (cache, dict(n=-1), EINVAL), (cache, dict(values=0), EINVAL), (cache, dict(dtype=5), EINVAL), (cache, dict(nslots=-1), EINVAL),
    (cache, dict(slots=None, nslots=2), EINVAL), (cache, dict(entries=None, nentries=2), EINVAL),
    # required pointers
    *[(f, {k: None}, EINVAL) for f, ks in ((scan, ("x", "gate", "weight", "y")), (scan_bwd, ("dy", "dx", "dgate")),
                                           (step, ("x", "gate", "h", "y")), (norm, ("x", "z", "y")), (norm_bwd, ("dy", "dx")),
                                           (cache, ("h", "q", "scale"))) for k in ks],
    # alignment
    (scan, dict(x=fake(1) + 1), EALIGN), (scan, dict(weight=fake(5) + 2), EALIGN), (scan, dict(h_in=fake(6) + 2), EALIGN),
    (scan_bwd, dict(workspace=fake(31) + 16), EALIGN), (step, dict(h=fake(6) + 2), EALIGN), (norm, dict(bias=fake(4) + 1), EALIGN),
    (cache, dict(h=fake(3) + 2), EALIGN), (cache, dict(scale=fake(5) + 1), EALIGN), (cache, dict(slots=fake(1) + 2), EALIGN),
    # overlaps
    (scan, dict(y=fake(1)), EINVAL), (scan, dict(y=fake(2) + 8), EINVAL), (scan, dict(h_out=fake(6) + 8), EINVAL),
    (scan, dict(h_out=fake(7)), EINVAL), (scan, dict(workspace=fake(4)), EINVAL), (scan_bwd, dict(dx=fake(9)), EINVAL),
    (scan_bwd, dict(dgate=fake(11)), EINVAL), (scan_bwd, dict(dh_in=fake(10)), EINVAL), (scan_bwd, dict(workspace=fake(13)), EINVAL),
    (step, dict(y=fake(6)), EINVAL), (step, dict(y=fake(1)), EINVAL), (norm, dict(y=fake(1)), EINVAL), (norm, dict(y=fake(2)), EINVAL),
    (norm_bwd, dict(dz=fake(7)), EINVAL), (norm_bwd, dict(dx=fake(6)), EINVAL), (cache, dict(q=fake(3) + 100), EINVAL),
    (cache, dict(scale=fake(4)), EINVAL), (cache, dict(h=fake(1)), EINVAL),
    (scan, dict(x_row=100, y=fake(1) + 2 * 100 * 15), EINVAL),      # inside the last rows of a strided x
    # workspaces
    (scan, dict(batch=1, seqlen=4096, workspace=None, workspace_bytes=0), EWORKSPACE), (scan, dict(workspace=None, workspace_bytes=0), OK),
    (scan_bwd, dict(workspace=None, workspace_bytes=0), EWORKSPACE), (scan_bwd, dict(workspace_bytes=64), EWORKSPACE),
    (norm_bwd, dict(workspace_bytes=16), EWORKSPACE),
]
RUNS = {m3.GatedScanArgs: ("gated_scan_fwd",), m3.GroupnormArgs: ("groupnorm_fwd",), m3.StateCacheArgs: ("state_store", "state_load")}


@pytest.mark.parametrize("i", range(len(CASES)))
def test_validation(lib, i):  # noqa: F811
    make, over, want = CASES[i]
    a = make(**over)
    assert getattr(lib, f"mamba3_{NAMES[type(a)]}_validate")(ctypes.byref(a)) == want, (NAMES[type(a)], over)
    if want != OK:      # the entry point refuses the same before any HIP call
        for run in RUNS.get(type(a), (NAMES[type(a)],)):
            assert getattr(lib, f"mamba3_{run}")(ctypes.byref(a), None) == want


def test_workspace_sizes(lib):  # noqa: F811
    size = lambda a: getattr(lib, f"mamba3_{NAMES[type(a)]}_workspace_size")(ctypes.byref(a))   # noqa: E731
    assert size(scan()) == 0 and size(scan(seqlen=4096)) > 0 and size(scan(batch=512, seqlen=4096, dim=64)) == 0
    assert size(scan(seqlen=4096, form=7)) == 0 and size(scan_bwd(fwd_form=7)) == 0
    assert size(scan_bwd()) > 0 and size(scan_bwd(fwd_seqlen=1 << 12)) > size(scan_bwd())
    assert size(norm_bwd()) > 0 and size(norm_bwd(dweight=None)) > 0 and size(norm_bwd(dweight=None, dbias=None)) == 0
    assert size(norm_bwd(fwd_groups=7)) == 0


MOST = (1 << 24) - 1


def ceil(a, b):
    return -(-a // b)


def apart(lib, a, want):  # noqa: F811
    """The validation's answer with arrays 2^42 bytes apart, so that none overlap whatever their sizes."""
    n, inner = 0, getattr(a, "fwd", None)
    for s in (inner, a) if inner is not None else (a,):
        for f, t in s._fields_:
            if t is ctypes.c_void_p and getattr(s, f):
                n += 1
                setattr(s, f, 0x1000000000000 + n * (1 << 42))
    if hasattr(a, "workspace_bytes"):
        a.workspace_bytes = 1 << 41
    assert getattr(lib, f"mamba3_{NAMES[type(a)]}_validate")(ctypes.byref(a)) == want


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_documented_workgroups(lib, dtype):  # noqa: F811
    """The header's formulas decide, at the last size taken and the first refused."""
    run = 32
    for dim in (1, 2, 63, 64, 129, 1000, 4096):      # (whole sequences of two tokens: nothing is cut)
        tiles = ceil(dim, 64 if dim % 2 else 128)
        for b in (MOST // tiles, MOST // tiles + 1):
            if b * 2 <= 1 << 30:
                apart(lib, scan(batch=b, seqlen=2, dim=dim, dtype=dtype), OK if b * tiles <= MOST else EINVAL)
        most = MOST // max(tiles, ceil(dim, 64))
        for b in (most, most + 1):
            apart(lib, scan_bwd(fwd_batch=b, fwd_seqlen=2, fwd_dim=dim, fwd_dtype=dtype), OK if b == most else EINVAL)
        for n in (MOST // tiles, MOST // tiles + 1):       # runs of one sequence
            if n * run <= 1 << 30:
                apart(lib, scan_bwd(fwd_batch=1, fwd_seqlen=n * run, fwd_dim=dim, fwd_dtype=dtype), OK if n * tiles <= MOST else EINVAL)
                apart(lib, scan_bwd(fwd_batch=1, fwd_seqlen=(n - 5) * run, fwd_dim=dim, fwd_dtype=dtype, fwd_cu_seqlens=fake(20), fwd_nseq=5),
                      OK if n * tiles <= MOST else EINVAL)
        quads = ceil(dim, 4)
        for b in (MOST * 256 // quads, MOST * 256 // quads + 1):
            if b < 1 << 31:
                apart(lib, step(batch=b, dim=dim, dtype=dtype), OK if ceil(b * quads, 256) <= MOST else EINVAL)
    apart(lib, norm(rows=(1 << 31) - 1, groups=100, dim=400, dtype=dtype), OK)
    for values in (1, 2048, 2049, 1 << 20):
        per = ceil(values, 4096 if dtype == BF16 else 2048)
        for n in (MOST // per, MOST // per + 1):
            apart(lib, cache(n=n, values=values, nslots=9, nentries=9, dtype=dtype), OK if n * per <= MOST else EINVAL)


def test_binding_refuses():
    x, w = torch.zeros(1, 4, 8), torch.zeros(8)
    for call in (lambda: m3.mamba3_gated_scan_fwd(x, x, w), lambda: m3.mamba3_gated_scan_bwd(x, x, w, dy=x),
                 lambda: m3.mamba3_gated_step(x[0], x[0], w, h=torch.zeros(4, 8)), lambda: m3.mamba3_groupnorm_fwd(x, w, groups=2),
                 lambda: m3.mamba3_groupnorm_bwd(x, w, dy=x, groups=2), lambda: m3.mamba3_state_store(torch.zeros(3, 4)),
                 lambda: m3.mamba3_state_load(torch.zeros(3, 4, dtype=torch.int8), torch.zeros(3, 1), h=torch.zeros(3, 4))):
        with pytest.raises(ValueError, match="device memory"):
            call()
    with pytest.raises(ValueError, match="dimensions"):
        m3.mamba3_gated_scan_fwd(x[0], x[0], w)
    with pytest.raises(ValueError, match="act must be"):
        m3.mamba3_groupnorm_fwd(x, w, groups=2, act="relu")
    with pytest.raises(ValueError, match="dy must have shape"):
        m3.mamba3_groupnorm_bwd(x, w, dy=x[0], groups=2)
    with pytest.raises(ValueError, match="kind must be"):
        m3.mamba3_state_store(torch.zeros(3, 4), kind="int2")
    with pytest.raises(ValueError, match="come together"):
        m3.mamba3_state_store(torch.zeros(3, 4), q=torch.zeros(3, 4, dtype=torch.int8))
