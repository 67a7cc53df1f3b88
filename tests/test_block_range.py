"""The norms and their gradients on rows far from unit size, against the fp64
definitions of oracle/block_oracle.py: with the squares inside fp32's range the
gradients are, whatever the powers of the root would be."""
import pytest

from oracle import block_oracle as K
from test_block_gpu import (EPS, Guard, _gpu, close, dev, f64, norm_in_inputs, norm_out_inputs, say, ssd,  # noqa: F401
                            torch_type)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# Row sizes, one row after the other, with their eps.  The cube of the root leaves
# fp32's normal range from rows of 4e12 on (k^3 < 2^-126), and its range below
# 1.4e-13 with eps = 0 (k^3 > 2^128).  The squares stay inside it: 32768 values of
# 10 x 1e16 have a sum of 3.3e38 < 2^128, and a square of 1e-15 is 1e-30, eight
# digits above the smallest normal value.
SIZES = [((1e14, 1.0, 1e16), EPS), ((1e-13, 1.0, 1e-15), 0.0)]


def sized(t, sizes, dim):
    """Indices 0, 1, .. of dimension dim times sizes[0], sizes[1], .. and over again."""
    f = torch.tensor([sizes[i % len(sizes)] for i in range(t.shape[dim])], device=t.device)
    return t * f.view([-1 if i == dim else 1 for i in range(t.dim())])


ROWS = [(5, 7, "f32"), (7, 64, "bf16"), (33, 1024, "bf16"), (4, 3, "f32"), (3, 500, "f32"), (4, 4096, "bf16"),
        (3, 9001, "bf16"), (3, 16384, "f32"), (300, 64, "bf16")]


@pytest.mark.parametrize("sizes,eps", SIZES)
@pytest.mark.parametrize("R,E,dtype", ROWS)
def test_norm_in_sizes(ssd, R, E, dtype, sizes, eps):  # noqa: F811
    r, p, s, w, du, _ = norm_in_inputs(R, E, dtype, 41)
    r = sized(r, sizes, 0)
    say("norm in", R, E, dtype, sizes, eps)
    args = [f64(r), None, None, f64(w), eps]
    u = ssd.norm_in(r, None, None, w, eps, dtype=torch_type(dtype))[1]
    close(u, K.norm_in(*args)[1], K.norm_in_bound(*args, dtype)[1], "u")
    args = [f64(v) for v in (du, None, r, p, s, w)] + [eps]
    got = ssd.norm_in_backward(du, None, r, p, s, w, eps)
    for name, v, want, bound in zip(("dr", "dp", "dw", "ds"), got, K.norm_in_backward(*args),
                                    K.norm_in_backward_bound(*args)):
        close(v, want, bound, name)


OUT = [(3, 2, 5, 7, 1, "f32"), (1, 16, 33, 64, 1, "bf16"), (2, 16, 7, 64, 16, "f32"), (2, 9, 5, 3, 3, "bf16"),
       (1, 64, 4, 64, 2, "bf16"), (2, 2, 3, 4999, 1, "f32"), (1, 1200, 3, 3, 2, "bf16")]


@pytest.mark.parametrize("sizes,eps", SIZES)
@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("B,H,N,d,groups,dtype", OUT)
def test_norm_out_sizes(ssd, B, H, N, d, groups, dtype, first, sizes, eps):  # noqa: F811
    y, z, w, do = norm_out_inputs(B, H, N, d, dtype, 42)
    y = sized(y, sizes, 2)
    say("norm out", B, H, N, d, groups, dtype, first, sizes, eps)
    args = [f64(v) for v in (y, z, w)] + [groups, first, eps]
    o = ssd.norm_out(y, z, w, eps, groups=groups, gate_first=first)
    close(o, K.norm_out(*args), K.norm_out_bound(*args, dtype), "o")
    args = [f64(v) for v in (do, y, z, w)] + [groups, first, eps]
    got = ssd.norm_out_backward(do, y, z, w, eps, groups=groups, gate_first=first)
    for name, v, want, bound in zip(("dy", "dz", "dw"), got, K.norm_out_backward(*args),
                                    K.norm_out_backward_bound(*args)):
        close(v, want, bound, name)


# From 2048 rows on a row of 513 to 1024 channels belongs to one wave forwards.
MANY = [(1, 16, 2100, 64, 1, "bf16"), (2, 16, 1024, 64, 1, "f32"), (1, 32, 1031, 64, 2, "bf16"),
        (2100, 11, 1, 60, 1, "bf16"), (3, 17, 700, 33, 1, "f32"), (1, 8, 2047, 128, 1, "bf16"),
        (1, 1, 2050, 1023, 1, "bf16")]


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("B,H,N,d,groups,dtype", MANY)
def test_norm_out_many_rows(ssd, B, H, N, d, groups, dtype, first):  # noqa: F811
    y, z, w, _ = norm_out_inputs(B, H, N, d, dtype, 43)
    say("norm out", B, H, N, d, groups, dtype, first)
    out = Guard()
    o = out.empty((B, N, H * d), torch_type(dtype))
    ssd.norm_out(y, z, w, EPS, groups=groups, gate_first=first, out=o)
    torch.cuda.synchronize()
    out.check()
    args = [f64(v) for v in (y, z, w)] + [groups, first, EPS]
    close(o, K.norm_out(*args), K.norm_out_bound(*args, dtype), "o")
