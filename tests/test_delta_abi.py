"""Host-side checks of include/hla_delta.h and of the Python calls over it (no GPU)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import higher_order_linear_chunked_b200 as hla
from higher_order_linear_chunked_b200 import delta

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "hla_delta.h")
NULL, SHAPE, ALIGN, DTYPE, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 5, 6


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(hla.LIB_PATH):
        from higher_order_linear_chunked_b200 import build
        build.build()
    return delta._library()


def test_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(hla_\w+)\s*\(", text))
    assert names == set(delta.EXPORTS)
    for n in names:
        assert hasattr(lib, n)
    assert lib.hla_delta_abi_version() == 1


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "use.c"
    src.write_text('#include "hla_delta.h"\nint main(void) { return HLA_BTHD == 1 && HLA_NORM_SILU == 2 ? 0 : 1; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-c", str(src), "-o",
                    str(tmp_path / "use.o")], check=True)


def test_sizes(lib):
    ws = lib.hla_delta_workspace_bytes
    for dtype in (hla.HLA_F32, hla.HLA_BF16):
        for d in (32, 64, 128):
            for dv in (32, 64, 128):
                assert 0 < ws(dtype, 1, 2, 4, 1, d, dv) <= ws(dtype, 1, 2, 4, 16384, d, dv)
                assert lib.hla_delta_kernel_launches(dtype, 1, 2, 4, 100, d, dv) >= 1
    for bad in ((7, 1, 1, 1, 1, 64, 64), (0, 0, 1, 1, 1, 64, 64), (0, 1, 0, 1, 1, 64, 64), (0, 1, 1, 1, 0, 64, 64),
                (0, 1, 2, 3, 1, 64, 64), (0, 1, 1, 1, 1, 48, 64), (0, 1, 1, 1, 1, 64, 256), (0, 8192, 4096, 4096, 1, 64, 64),
                (0, 1 << 15, 1, 1, 1 << 16, 64, 64)):
        assert ws(*bad) == 0 and lib.hla_delta_kernel_launches(*bad) == 0
    nb = lib.hla_group_norm_backward_workspace_bytes
    assert nb(0, 1, 64, 2) == 2 * 64 * 4
    assert nb(1, 1 << 20, 1024, 16) > 0
    for bad in ((7, 1, 64, 2), (0, 0, 64, 2), (0, 1, 64, 3), (0, 1, 1024, 1), (0, 1, 0, 1), (0, 1 << 31, 64, 2),
                (0, 1 << 30, 64, 16)):
        assert nb(*bad) == 0, bad


def _forward(lib, **kw):
    a = dict(q=16, k=16, v=16, g=4, beta=4, state_in=0, lengths=0, o=16, state_out=0, B=1, Hk=1, H=2, T=8, d=64,
             dv=64, dtype=1, layout=0, scale=1.0, ws=16, wsb=1 << 40, stream=0)
    a.update(kw)
    return lib.hla_delta_forward(*a.values())


def test_forward_argument_errors(lib):
    for n in ("q", "k", "v", "g", "beta", "o"):
        assert _forward(lib, **{n: 0}) == NULL
    for n in ("q", "k", "v", "o", "state_in", "state_out", "ws"):
        assert _forward(lib, **{n: 24}) == ALIGN
    for n in ("g", "beta", "lengths"):
        assert _forward(lib, **{n: 6}) == ALIGN
    assert _forward(lib, B=0) == SHAPE and _forward(lib, T=0) == SHAPE and _forward(lib, Hk=3) == SHAPE
    assert _forward(lib, B=1 << 24) == SHAPE and _forward(lib, B=1 << 14, T=1 << 17) == SHAPE
    assert _forward(lib, dtype=2) == DTYPE
    assert _forward(lib, d=16) == UNSUPPORTED and _forward(lib, dv=96) == UNSUPPORTED
    assert _forward(lib, layout=2) == UNSUPPORTED
    assert _forward(lib, ws=0) == WORKSPACE and _forward(lib, wsb=8) == WORKSPACE


def test_step_argument_errors(lib):
    def step(**kw):
        a = dict(state=16, q=16, k=16, v=16, g=4, beta=4, o=16, B=1, Hk=1, H=2, d=64, dv=64, dtype=1, scale=1.0, s=0)
        a.update(kw)
        return lib.hla_delta_step(*a.values())
    for n in ("state", "q", "k", "v", "g", "beta", "o"):
        assert step(**{n: 0}) == NULL
    for n in ("state", "q", "k", "v", "o"):
        assert step(**{n: 8}) == ALIGN
    assert step(H=0) == SHAPE and step(Hk=3) == SHAPE and step(dtype=5) == DTYPE and step(d=65) == UNSUPPORTED


def test_backward_argument_errors(lib):
    ws = lib.hla_delta_backward_workspace_bytes
    for dtype in (hla.HLA_F32, hla.HLA_BF16):
        assert 0 < ws(dtype, 1, 2, 2, 1, 64, 64) <= ws(dtype, 1, 2, 2, 4096, 64, 64) < ws(dtype, 1, 1, 2, 4096, 64, 64)
    assert lib.hla_delta_backward_kernel_launches(1, 1, 1, 2, 100, 64, 64) == 5    # shared heads: one more
    assert lib.hla_delta_backward_kernel_launches(1, 1, 2, 2, 100, 64, 64) == 4
    assert ws(1, 1, 2, 3, 1, 64, 64) == 0 and lib.hla_delta_backward_kernel_launches(1, 1, 1, 1, 1, 8, 64) == 0

    def back(**kw):
        a = dict(q=16, k=16, v=16, g=4, beta=4, state_in=0, lengths=0, dout=16, dstate_out=0, dq=16, dk=16, dv_out=16,
                 dg=4, dbeta=4, dstate_in=0, B=1, Hk=1, H=2, T=8, d=64, dv=64, dtype=1, layout=0, scale=1.0, ws=16,
                 wsb=1 << 40, stream=0)
        a.update(kw)
        return lib.hla_delta_backward(*a.values())

    for n in ("q", "k", "v", "g", "beta", "dout", "dq", "dk", "dv_out", "dg", "dbeta"):
        assert back(**{n: 0}) == NULL, n
    for n in ("q", "k", "v", "dout", "dq", "dk", "dv_out", "state_in", "dstate_out", "dstate_in", "ws"):
        assert back(**{n: 8}) == ALIGN, n
    for n in ("g", "beta", "dg", "dbeta", "lengths"):
        assert back(**{n: 2}) == ALIGN, n
    assert back(H=0) == SHAPE and back(dtype=3) == DTYPE and back(dv=16) == UNSUPPORTED and back(layout=7) == UNSUPPORTED
    assert back(ws=0) == WORKSPACE and back(wsb=1024) == WORKSPACE


def test_norm_argument_errors(lib):
    def fwd(**kw):
        a = dict(x=16, gate=0, w=4, b=4, y=16, rows=3, C=64, groups=2, dtype=0, eps=1e-5, flags=0, s=0)
        a.update(kw)
        return lib.hla_group_norm_forward(*a.values())

    def bwd(**kw):
        a = dict(x=16, gate=16, w=4, b=4, dy=16, dx=16, dgate=16, dw=4, db=4, rows=3, C=64, groups=2, dtype=0,
                 eps=1e-5, flags=0, ws=16, wsb=1 << 30, s=0)
        a.update(kw)
        return lib.hla_group_norm_backward(*a.values())

    assert fwd(x=0) == NULL and fwd(y=0) == NULL
    assert fwd(gate=8) == ALIGN and fwd(w=2) == ALIGN
    assert bwd(x=0) == NULL and bwd(dy=0) == NULL and bwd(dx=0) == NULL and bwd(dgate=0) == NULL
    assert bwd(gate=0) == UNSUPPORTED                       # a gate's gradient without a gate
    assert bwd(dgate=8) == ALIGN and bwd(db=1) == ALIGN and bwd(ws=8) == ALIGN
    assert bwd(ws=0) == WORKSPACE and bwd(wsb=16) == WORKSPACE
    for f in (fwd, bwd):
        assert f(rows=0) == SHAPE and f(groups=3) == SHAPE and f(dtype=9) == DTYPE and f(flags=4) == UNSUPPORTED
        assert f(C=1026, groups=2) == UNSUPPORTED           # 513 channels in a group


def test_python_refusals_name_the_argument():
    q = torch.zeros(1, 1, 4, 64)
    g = torch.zeros(1, 1, 4)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        hla.gated_delta(q, q, q, g, g)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        hla.gated_delta_step(torch.zeros(1, 1, 64, 64), q[:, :, 0], q[:, :, 0], q[:, :, 0], g[:, :, 0], g[:, :, 0])
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        hla.group_norm(q, 2)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        hla.group_norm_backward(q, q, 2)
    assert hla.gated_delta_workspace_bytes(torch.float16, 1, 1, 1, 1, 64, 64) == 0
