"""Host-side checks of the gated delta rule's and the layer norm's C ABI: sizes
and argument errors, reported before any CUDA call."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from gated_linear_recurrence_b200 import build
    build.build()
    from gated_linear_recurrence_b200 import esa
    return esa.load_library()


def P(x):
    return ctypes.c_void_p(x) if x else None


def _fwd(lib, q=0x1000, k=0x2000, ldqk=128, v=0x3000, ldv=128, a=0x4002, b=0x5002, ldg=2, y=0x6000, S=0, B=2, T=8,
         H=2, D=64, scale=0.1, S0=0, dtype=1, keep=1, ws=0x10000, wsb=1 << 40):
    return lib.esa_delta_fwd(P(q), P(k), ldqk, P(v), ldv, P(a), P(b), ldg, P(y), P(S), B, T, H, D, scale, P(S0), dtype,
                             keep, P(ws), wsb, None)


def test_delta_forward_errors(lib):
    from gated_linear_recurrence_b200 import esa
    assert _fwd(lib, dtype=4) == esa.ESA_ERR_ARG
    assert _fwd(lib, dtype=3) == esa.ESA_ERR_UNSUPPORTED
    for D in (8, 16, 48, 256):
        assert _fwd(lib, D=D, ldqk=2 * D, ldv=2 * D) == esa.ESA_ERR_UNSUPPORTED
    assert _fwd(lib, B=-1) == esa.ESA_ERR_ARG
    assert _fwd(lib, H=0) == esa.ESA_ERR_ARG
    assert _fwd(lib, keep=2) == esa.ESA_ERR_ARG
    assert _fwd(lib, scale=float("nan")) == esa.ESA_ERR_ARG
    assert _fwd(lib, scale=float("inf")) == esa.ESA_ERR_ARG
    for missing in ("q", "k", "v", "a", "b", "y"):
        assert _fwd(lib, **{missing: 0}) == esa.ESA_ERR_ARG
    for off in ("q", "k", "v", "y", "S", "S0", "ws"):
        assert _fwd(lib, **{off: 0x7008}) == esa.ESA_ERR_ALIGN
    assert _fwd(lib, a=0x4001) == esa.ESA_ERR_ALIGN
    assert _fwd(lib, ldqk=120) == esa.ESA_ERR_ARG
    assert _fwd(lib, ldv=132) == esa.ESA_ERR_ALIGN
    assert _fwd(lib, ldg=1) == esa.ESA_ERR_ARG
    assert _fwd(lib, ws=0) == esa.ESA_ERR_WORKSPACE
    assert _fwd(lib, wsb=16) == esa.ESA_ERR_WORKSPACE


def test_delta_backward_and_step_errors(lib):
    from gated_linear_recurrence_b200 import esa

    def bwd(dy=0x6000, dq=0x7000, dk=0x8000, dv=0x9000, da=0xa000, db=0xb000, wsb=1 << 40, ws=0x10000):
        return lib.esa_delta_bwd(P(0x1000), P(0x2000), 128, P(0x3000), 128, P(0x4000), P(0x5000), 2, P(dy), None, P(dq),
                                 P(dk), P(dv), P(da), P(db), None, 2, 8, 2, 64, 0.1, None, 1, P(ws), wsb, None)

    for n in ("dy", "dq", "dk", "dv", "da", "db"):
        assert bwd(**{n: 0}) == esa.ESA_ERR_ARG
    for n in ("dy", "dq", "dk", "dv", "ws"):
        assert bwd(**{n: 0x7004}) == esa.ESA_ERR_ALIGN
    assert bwd(da=0x7001) == esa.ESA_ERR_ALIGN
    assert bwd(wsb=lib.esa_delta_workspace_size(2, 8, 2, 64, 1, 1) - 1) == esa.ESA_ERR_WORKSPACE

    def step(S=0x6000, y=0x7000, D=64, dtype=1, q=0x1000):
        return lib.esa_delta_step(P(q), P(0x2000), 2 * D, P(0x3000), 2 * D, P(0x4000), P(0x5000), 2, P(S), P(y), 2, 2, D, 0.1,
                                  dtype, None)

    assert step(S=0) == esa.ESA_ERR_ARG
    assert step(y=0) == esa.ESA_ERR_ARG
    assert step(D=40) == esa.ESA_ERR_UNSUPPORTED
    assert step(dtype=3) == esa.ESA_ERR_UNSUPPORTED
    assert step(S=0x6004) == esa.ESA_ERR_ALIGN


def test_sizes(lib):
    assert lib.esa_delta_workspace_size(2, 100, 3, 24, 1, 1) == 0
    assert lib.esa_delta_workspace_size(-1, 100, 3, 64, 1, 1) == 0
    assert lib.esa_delta_workspace_size(2, 100, 3, 64, 3, 1) == 0
    assert 0 < lib.esa_delta_workspace_size(2, 100, 3, 64, 1, 0) < lib.esa_delta_workspace_size(2, 100, 3, 64, 1, 1)
    # beyond 32 bits
    assert lib.esa_delta_workspace_size(64, 65536, 8, 128, 1, 1) > 1 << 34
    assert lib.esa_norm_workspace_size(0, 16, 0, 0) > 0
    assert lib.esa_norm_workspace_size(10, 0, 0, 0) == 0
    assert lib.esa_norm_workspace_size(10, 16385, 0, 0) == 0
    assert lib.esa_norm_workspace_size(10, 16, 0, 1) == 0


def test_norm_errors(lib):
    from gated_linear_recurrence_b200 import esa

    def fwd(x=0x1000, ldx=64, r=0, ldr=64, w=0x3000, c=0x4000, y=0x5000, h=0, s=0, rows=4, N=64, eps=1e-5, dt=1, wdt=1):
        return lib.esa_norm_fwd(P(x), ldx, P(r), ldr, P(w), P(c), P(y), P(h), P(s), rows, N, eps, dt, wdt, None)

    assert fwd(rows=-1) == esa.ESA_ERR_ARG
    assert fwd(rows=1 << 31) == esa.ESA_ERR_ARG
    assert fwd(N=0) == esa.ESA_ERR_ARG
    assert fwd(N=20000, ldx=20000) == esa.ESA_ERR_UNSUPPORTED
    assert fwd(dt=3) == esa.ESA_ERR_UNSUPPORTED
    assert fwd(dt=1, wdt=2) == esa.ESA_ERR_UNSUPPORTED
    assert fwd(eps=-1.0) == esa.ESA_ERR_ARG
    assert fwd(eps=float("nan")) == esa.ESA_ERR_ARG
    assert fwd(ldx=63) == esa.ESA_ERR_ARG
    assert fwd(x=0) == esa.ESA_ERR_ARG
    assert fwd(y=0) == esa.ESA_ERR_ARG
    assert fwd(r=0x2000) == esa.ESA_ERR_ARG               # a residual without h
    assert fwd(r=0x2000, h=0x6000, ldr=10) == esa.ESA_ERR_ARG
    assert fwd(x=0x1001) == esa.ESA_ERR_ALIGN
    assert fwd(s=0x6004) == esa.ESA_ERR_ALIGN

    def bwd(dy=0x1000, h=0x2000, w=0x3000, s=0x4000, dh=0, dx=0x5000, dw=0x6000, dc=0x7000, ws=0x8000, wsb=1 << 30):
        return lib.esa_norm_bwd(P(dy), 64, P(h), 64, P(w), P(s), P(dh), 64, P(dx), P(dw), P(dc), 4, 64, 1, 1, P(ws), wsb,
                                None)

    for n in ("dy", "h", "s", "dx"):
        assert bwd(**{n: 0}) == esa.ESA_ERR_ARG
    assert bwd(ws=0) == esa.ESA_ERR_WORKSPACE
    assert bwd(wsb=8) == esa.ESA_ERR_WORKSPACE
    assert bwd(dx=0x5001) == esa.ESA_ERR_ALIGN


def test_no_device(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is present; this checks the device-less path")
    from gated_linear_recurrence_b200 import esa
    assert _fwd(lib) == esa.ESA_ERR_DEVICE
    assert lib.esa_norm_fwd(P(0x1000), 64, None, 64, None, None, P(0x2000), None, None, 4, 64, 1e-5, 1, 1,
                            None) == esa.ESA_ERR_DEVICE


def test_bindings_refuse_cpu_tensors(lib):
    import torch
    from gated_linear_recurrence_b200 import esa_delta_fwd, esa_delta_step, esa_norm_bwd, esa_norm_fwd
    z, g = torch.zeros(1, 4, 2, 32), torch.zeros(1, 4, 2)
    with pytest.raises(TypeError):
        esa_delta_fwd(z, z, z, g, g)
    with pytest.raises(TypeError):
        esa_delta_step(z[:, 0], z[:, 0], z[:, 0], g[:, 0], g[:, 0], torch.zeros(1, 2, 32, 32))
    with pytest.raises(TypeError):
        esa_norm_fwd(z)
    with pytest.raises(TypeError):
        esa_norm_bwd(z, z, None, torch.zeros(8, 2))
