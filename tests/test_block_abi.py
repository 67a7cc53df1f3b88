"""The gated recurrence's and the norms' calls on the CPU: bad arguments are
rejected before any HIP call (fake, never dereferenced addresses are passed;
no call here reaches a kernel launch), and empty inputs are valid."""
import math

import pytest

from mamba_ssd_sequence_amd import ssd

A = [0x10000000 * (i + 1) for i in range(24)]  # distinct, 16-byte aligned fake addresses
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return ssd.lib()


def scan(lib, *, x=A[0], Ap=A[1], Ip=A[2], h0=None, B=1, H=2, N=100, d=64, scale=2, dtype=1, y=A[4], hf=None, ws=A[6],
         wsb=BIG):
    return lib.ssd_gated_scan(x, Ap, Ip, h0, B, H, N, d, scale, dtype, y, hf, ws, wsb, None)


def test_scan_errors(lib):
    for name in ("x", "Ap", "y"):
        assert scan(lib, **{name: None}) == 1
    assert "NULL" in lib.ssd_last_error().decode()
    for bad in (dict(B=-1), dict(H=-1), dict(N=-1), dict(d=0), dict(d=-4), dict(B=BIG, H=BIG), dict(B=1 << 31),
                dict(H=1 << 20, N=1 << 20)):
        assert scan(lib, **bad) == 2, bad
    assert scan(lib, scale=3) == 3 and scan(lib, scale=-1) == 3
    assert scan(lib, dtype=2) == 3
    assert scan(lib, H=1, N=1, d=(1 << 20) + 1) == 3
    for name in ("x", "Ap", "Ip", "y", "h0", "hf", "ws"):
        assert scan(lib, **{name: A[8] + 4}) == 4, name
    assert scan(lib, y=A[0]) == 5 and scan(lib, y=A[2] + 64) == 5
    assert scan(lib, h0=A[5], hf=A[5]) == 5
    assert "final_state" in lib.ssd_last_error().decode()
    assert scan(lib, hf=A[4] + 16) == 5
    assert scan(lib, N=0, x=None, Ap=None, Ip=None, y=None, ws=None, wsb=0) == 0
    assert scan(lib, B=0, x=None, Ap=None, y=None) == 0
    assert scan(lib, N=0, h0=A[5], hf=A[5] + 16) == 5  # still checked
    assert scan(lib, N=0, scale=9) == 3


def test_scan_workspace(lib):
    size = lib.ssd_gated_scan_workspace_size
    bwd = lib.ssd_gated_scan_backward_workspace_size
    assert size(1, 1, -1, 64) == 0 and size(1, 1, 0, 64) == 0 and size(1, 1, 10, 0) == 0 and size(BIG, BIG, 1, 64) == 0
    for B, H, N, d in ((1, 1, 65536, 64), (1, 16, 65536, 64), (2, 3, 1000, 33), (4, 16, 2048, 64)):
        need, back = size(B, H, N, d), bwd(B, H, N, d)
        if need:
            assert scan(lib, B=B, H=H, N=N, d=d, wsb=need - 1) == 6
            assert scan(lib, B=B, H=H, N=N, d=d, ws=None, wsb=0) == 6
            assert scan(lib, B=B, H=H, N=N, d=d, ws=A[0]) == 5  # the workspace over an input
        if back:
            assert scan_bwd(lib, B=B, H=H, N=N, d=d, wsb=back - 1) == 6


def step(lib, *, x=A[0], Ap=A[1], Ip=None, st=A[3], S=2, H=2, d=64, scale=0, dtype=0, out=A[4]):
    return lib.ssd_gated_scan_step(x, Ap, Ip, st, S, H, d, scale, dtype, out, None)


def test_step_errors(lib):
    for name in ("x", "Ap", "st", "out"):
        assert step(lib, **{name: None}) == 1
    assert step(lib, S=-1) == 2 and step(lib, d=0) == 2 and step(lib, S=BIG, H=BIG) == 2
    assert step(lib, scale=4) == 3 and step(lib, dtype=-1) == 3
    assert step(lib, st=A[3] + 8) == 4
    assert step(lib, out=A[0]) == 5
    assert step(lib, out=A[3] + 16) == 5  # over the state, but not the state itself
    assert step(lib, x=A[3], st=A[3], out=A[3]) == 5  # in place over the input
    assert step(lib, S=0, x=None, Ap=None, st=None, out=None) == 0


def scan_bwd(lib, *, x=A[0], Ap=A[1], Ip=A[2], h0=None, y=A[3], dy=A[4], dl=None, B=1, H=2, N=100, d=64, scale=2,
             dtype=1, dx=A[5], dA=A[6], dI=A[7], d0=None, ws=A[8], wsb=BIG):
    return lib.ssd_gated_scan_backward(x, Ap, Ip, h0, y, dy, dl, B, H, N, d, scale, dtype, dx, dA, dI, d0, ws, wsb, None)


def test_scan_backward_errors(lib):
    for name in ("x", "Ap", "y", "dy", "dx", "dA"):
        assert scan_bwd(lib, **{name: None}) == 1, name
    assert scan_bwd(lib, Ip=None) == 1 and scan_bwd(lib, dI=None) == 1
    assert scan_bwd(lib, N=-1) == 2 and scan_bwd(lib, d=0) == 2
    assert scan_bwd(lib, scale=3) == 3 and scan_bwd(lib, dtype=5) == 3
    for name in ("dx", "dA", "dI", "y", "dy", "dl", "d0", "h0", "ws"):
        assert scan_bwd(lib, **{name: A[9] + 8}) == 4, name
    assert scan_bwd(lib, dx=A[4]) == 5 and scan_bwd(lib, dA=A[5]) == 5 and scan_bwd(lib, d0=A[3]) == 5
    assert scan_bwd(lib, N=0, x=None, Ap=None, Ip=None, y=None, dy=None, dx=None, dA=None, dI=None) == 0
    assert scan_bwd(lib, N=0, dl=A[9], d0=A[9]) == 5


def norm_in(lib, *, r=A[0], p=A[1], s=A[2], w=A[3], rows=5, E=64, eps=1e-5, dtype=1, ro=A[4], u=A[5]):
    return lib.ssd_norm_in(r, p, s, w, rows, E, eps, dtype, ro, u, None)


def test_norm_in_errors(lib):
    for name in ("r", "w", "u", "ro", "p"):
        assert norm_in(lib, **{name: None}) == 1, name
    assert norm_in(lib, p=None, ro=None) == 1  # a scale without a branch
    assert norm_in(lib, rows=-1) == 2 and norm_in(lib, E=0) == 2 and norm_in(lib, rows=1 << 60, E=64) == 2
    assert norm_in(lib, E=32769) == 3 and norm_in(lib, dtype=2) == 3
    for eps in (-1e-6, math.nan, math.inf):
        assert norm_in(lib, eps=eps) == 3
    assert norm_in(lib, u=A[5] + 2) == 4 and norm_in(lib, s=A[2] + 4) == 4
    assert norm_in(lib, ro=A[0]) == 5 and norm_in(lib, u=A[1]) == 5 and norm_in(lib, u=A[4] + 16) == 5
    assert norm_in(lib, rows=0, r=None, p=None, s=None, w=None, ro=None, u=None) == 0


def norm_in_bwd(lib, *, du=A[0], dro=A[1], r=A[2], p=A[3], s=A[4], w=A[5], rows=5, E=64, eps=1e-5, dtype=1, dr=A[6],
                dp=A[7], dw=A[8], ds=A[9], ws=A[10], wsb=BIG):
    return lib.ssd_norm_in_backward(du, dro, r, p, s, w, rows, E, eps, dtype, dr, dp, dw, ds, ws, wsb, None)


def test_norm_in_backward_errors(lib):
    for name in ("du", "r", "w", "dr", "dw", "p", "s", "dp", "ds"):
        assert norm_in_bwd(lib, **{name: None}) == 1, name
    assert norm_in_bwd(lib, rows=-1) == 2 and norm_in_bwd(lib, E=1 << 16) == 3 and norm_in_bwd(lib, dtype=9) == 3
    assert norm_in_bwd(lib, eps=-1.0) == 3
    need = lib.ssd_norm_in_backward_workspace_size(5, 64)
    assert need > 0 and norm_in_bwd(lib, wsb=need - 1) == 6 and norm_in_bwd(lib, ws=None) == 6
    assert lib.ssd_norm_in_backward_workspace_size(0, 64) == 0
    assert lib.ssd_norm_in_backward_workspace_size(5, 0) == 0 and lib.ssd_norm_in_backward_workspace_size(-5, 4) == 0
    assert norm_in_bwd(lib, dr=A[6] + 4) == 4 and norm_in_bwd(lib, dr=A[1]) == 5 and norm_in_bwd(lib, ds=A[8]) == 5


def norm_out(lib, *, y=A[0], z=A[1], w=A[2], B=2, H=4, N=10, d=64, groups=1, first=1, eps=1e-5, dtype=1, o=A[3]):
    return lib.ssd_norm_out(y, z, w, B, H, N, d, groups, first, eps, dtype, o, None)


def test_norm_out_errors(lib):
    for name in ("y", "z", "w", "o"):
        assert norm_out(lib, **{name: None}) == 1, name
    for bad in (dict(B=-1), dict(N=-1), dict(H=0), dict(d=0), dict(groups=0), dict(groups=3), dict(groups=8),
                dict(B=BIG, N=BIG)):
        assert norm_out(lib, **bad) == 2, bad
    assert norm_out(lib, first=2) == 3 and norm_out(lib, dtype=2) == 3 and norm_out(lib, eps=-0.5) == 3
    assert norm_out(lib, H=1024, d=64) == 3  # 65536 channels in one group
    assert norm_out(lib, z=A[1] + 2) == 4
    assert norm_out(lib, o=A[1]) == 5 and norm_out(lib, o=A[0] + 128) == 5
    assert norm_out(lib, B=0, y=None, z=None, w=None, o=None) == 0


def norm_out_bwd(lib, *, do=A[0], y=A[1], z=A[2], w=A[3], B=2, H=4, N=10, d=64, groups=1, first=1, eps=1e-5, dtype=1,
                 dy=A[4], dz=A[5], dw=A[6], ws=A[7], wsb=BIG):
    return lib.ssd_norm_out_backward(do, y, z, w, B, H, N, d, groups, first, eps, dtype, dy, dz, dw, ws, wsb, None)


def test_norm_out_backward_errors(lib):
    for name in ("do", "y", "z", "w", "dy", "dz", "dw"):
        assert norm_out_bwd(lib, **{name: None}) == 1, name
    assert norm_out_bwd(lib, groups=3) == 2 and norm_out_bwd(lib, first=-1) == 3 and norm_out_bwd(lib, dtype=3) == 3
    need = lib.ssd_norm_out_backward_workspace_size(2, 4, 10, 64, 1)
    assert need > 0 and norm_out_bwd(lib, wsb=need - 1) == 6
    assert lib.ssd_norm_out_backward_workspace_size(2, 4, 10, 64, 3) == 0
    assert norm_out_bwd(lib, dw=A[6] + 4) == 4 and norm_out_bwd(lib, dz=A[4]) == 5 and norm_out_bwd(lib, dy=A[3]) == 5


def test_binding_refuses():
    torch = pytest.importorskip("torch")
    x = torch.zeros(1, 2, 3, 4)
    with pytest.raises(ValueError):
        ssd.gated_scan(x, x, scale=0)
    with pytest.raises(ValueError):
        ssd.norm_in(x, x, None, torch.ones(4), 1e-5)
    with pytest.raises(ValueError):
        ssd.norm_out(x, torch.zeros(1, 3, 8), torch.ones(8), 1e-5)
    with pytest.raises(TypeError):
        ssd.gated_scan_step(None, x, None, x, scale=0)
