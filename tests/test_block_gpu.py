"""The gated linear recurrence and the norms around a mixer block on the GPU,
against the fp64 definitions of oracle/block_oracle.py.  Every element is held
to the oracle's bound on an fp32 evaluation (bf16 outputs: half a bf16 step
more)."""
import numpy as np
import pytest

from oracle import block_oracle as K

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

EPS = 1e-5
SCALES = (K.PLAIN, K.CONVEX, K.UNIT)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.fixture(scope="module")
def ssd():
    from mamba_ssd_sequence_amd import ssd
    ssd.lib()
    return ssd


def say(*a):
    print(*a, flush=True)


def torch_type(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def dev(v, dtype="f32"):
    return None if v is None else torch.from_numpy(np.ascontiguousarray(v)).to(torch_type(dtype)).cuda()


def f64(t):
    return None if t is None else t.double().cpu().numpy()


class Guard:
    """Output tensors between guard elements that a call must leave alone."""

    def __init__(self):
        self.all = []

    def empty(self, shape, dtype=torch.float32):
        n = int(np.prod(shape))
        buf = torch.full((n + 512,), 77.0, dtype=dtype, device="cuda")
        self.all.append((buf, n))
        buf[256:256 + n] = float("nan")
        return buf[256:256 + n].view(shape)

    def check(self):
        for buf, n in self.all:
            assert bool((buf[:256] == 77).all()) and bool((buf[256 + n:] == 77).all())


def garbage(nbytes):
    """A workspace full of NaN."""
    return torch.full((max(nbytes, 16),), 255, dtype=torch.uint8, device="cuda")


def close(got, want, bound, name):
    got = f64(got)
    assert got.shape == want.shape, name
    ok = np.isfinite(want)
    assert (np.isnan(got) == np.isnan(want)).all(), name
    assert (got[~ok & ~np.isnan(want)] == want[~ok & ~np.isnan(want)]).all(), name
    worst = float((np.abs(got - want)[ok] / bound[ok]).max()) if ok.any() else 0.0
    say(f"  {name}: {worst:.3g} of the bound")
    assert worst <= 1, (name, worst)


# ---- the recurrence ----


def scan_inputs(B, H, N, d, dtype, gate, init, seed, packed=False):
    g = np.random.default_rng(seed)
    x, A, I = g.standard_normal((3, B, H, N, d))
    A -= 3
    if packed:  # sequences that start inside the row, and tokens that leave the state alone
        A[:, :, g.random(N) < 0.1] = np.inf
        A[:, :, g.random(N) < 0.1] = -np.inf
    t = [dev(x, dtype), dev(A, dtype), dev(I, dtype) if gate else None]
    h0 = dev(g.standard_normal((B, H, d)).astype(np.float32)) if init else None
    return t, h0, g


def bounded_scan(ssd, t, h0, scale, seed_state=True):
    B, H, N, d = t[0].shape
    out = Guard()
    y, last = out.empty((B, H, N, d)), out.empty((B, H, d))
    ws = garbage(ssd.lib().ssd_gated_scan_workspace_size(B, H, N, d))
    got = ssd.gated_scan(*t, scale=scale, initial_state=h0, final_state=last, y=y, workspace=ws)
    assert got is y
    torch.cuda.synchronize()
    out.check()
    return y, last


def bounded_backward(ssd, t, h0, y, dy, dl, scale):
    """ssd_gated_scan_backward into guarded outputs"""
    B, H, N, d = t[0].shape
    out = Guard()
    dx, dA = out.empty(y.shape), out.empty(y.shape)
    dI = out.empty(y.shape) if t[2] is not None else None
    d0 = out.empty((B, H, d))
    need = ssd.lib().ssd_gated_scan_backward_workspace_size(B, H, N, d)
    ws = garbage(need)
    p = ssd._ptr
    ssd._check(ssd.lib().ssd_gated_scan_backward(
        p(t[0]), p(t[1]), p(t[2]), p(h0), p(y), p(dy), p(dl), B, H, N, d, scale,
        1 if t[0].dtype == torch.bfloat16 else 0, p(dx), p(dA), p(dI), p(d0), p(ws), need,
        ssd._stream(t[0].device)))
    torch.cuda.synchronize()
    out.check()
    return dx, dA, dI, d0


SCAN = [
    # B, H, N, d, dtype, gate, init, packed
    (1, 1, 1, 1, "f32", False, False, False),
    (1, 2, 1, 64, "bf16", True, True, False),
    (2, 1, 3, 3, "bf16", True, True, False),
    (1, 2, 31, 64, "f32", True, False, False),
    (2, 2, 33, 32, "bf16", False, True, True),
    (1, 3, 129, 65, "bf16", True, True, True),
    (1, 1, 257, 16, "f32", True, True, True),
    (1, 2, 511, 128, "bf16", True, False, False),
    (1, 1, 513, 20, "bf16", True, True, False),
    (3, 2, 1000, 33, "f32", True, True, True),
    (1, 2, 1025, 36, "f32", False, True, False),
    (2, 3, 2049, 64, "bf16", True, True, True),
    (1, 1, 4100, 200, "bf16", True, True, False),
    (40, 16, 70, 64, "bf16", True, True, True),
    (1, 1, 9000, 64, "f32", True, True, False),
    # many tiles a head, shared out: spans of them, in workgroups of 8 and of 16 waves
    (1, 1, 40000, 3, "bf16", True, True, False),
    (1, 14, 20000, 32, "bf16", False, True, True),
    (1, 12, 12000, 64, "f32", True, True, False),
    # heads whose last piece or slab is moved back: 4 n + 1 .. 3 channels, one more than a slab, more slabs than even
    (1, 2, 300, 5, "bf16", True, True, False),
    (2, 1, 300, 34, "bf16", True, True, True),
    (1, 1, 700, 67, "f32", True, True, False),
    (1, 1, 130, 1217, "bf16", True, True, False),
    (1, 2, 600, 2, "f32", True, True, False),
    # heads enough to take a head's tiles one after the other
    (65, 8, 600, 64, "bf16", True, True, True),
    (65, 8, 300, 17, "f32", False, True, False),
]


@pytest.mark.parametrize("B,H,N,d,dtype,gate,init,packed", SCAN)
def test_scan(ssd, B, H, N, d, dtype, gate, init, packed):
    for scale in SCALES:
        t, h0, _ = scan_inputs(B, H, N, d, dtype, gate, init, 3, packed)
        say("scan", B, H, N, d, dtype, gate, init, packed, scale)
        y, last = bounded_scan(ssd, t, h0, scale)
        args = [f64(v) for v in t] + [f64(h0), scale]
        want, bound = K.scan(*args), K.scan_bound(*args)
        close(y, want, bound, "y")
        close(last, want[:, :, -1], bound[:, :, -1], "last")
        assert torch.equal(last, y[:, :, -1])


@pytest.mark.parametrize("B,H,N,d,dtype,gate,init,packed", SCAN)
def test_scan_backward(ssd, B, H, N, d, dtype, gate, init, packed):
    for scale in SCALES:
        t, h0, g = scan_inputs(B, H, N, d, dtype, gate, init, 4, packed)
        args = [f64(v) for v in t] + [f64(h0)]
        y = dev(K.scan(*args, scale).astype(np.float32))
        dy = dev(g.standard_normal((B, H, N, d)).astype(np.float32))
        dl = dev(g.standard_normal((B, H, d)).astype(np.float32)) if init else None
        say("scan backward", B, H, N, d, dtype, gate, init, packed, scale)
        got = bounded_backward(ssd, t, h0, y, dy, dl, scale)
        args += [f64(y), f64(dy), f64(dl), scale]
        for name, v, want, bound in zip(("dx", "dA", "dI", "dh0"), got, K.scan_backward(*args),
                                        K.scan_backward_bound(*args)):
            if v is not None:
                close(v, want, bound, name)
        # the binding returns the same
        again = ssd.gated_scan_backward(*t, y, dy, scale=scale, initial_state=h0, d_final_state=dl)
        for a, b in zip(got[:3] + ((got[3],) if init else (None,)), again):
            assert (a is None) == (b is None) and (a is None or torch.equal(a, b))


@pytest.mark.parametrize("d", [64, 33])
def test_scan_long_memory(ssd, d):
    """Decays within 1e-4 of one: the state remembers thousands of tokens."""
    g = np.random.default_rng(5)
    N = 6000
    t = [dev(g.standard_normal((1, 1, N, d))), dev(g.standard_normal((1, 1, N, d)) - 9), None]
    for scale in SCALES:
        y, _ = bounded_scan(ssd, t, None, scale)
        args = [f64(v) for v in t] + [None, scale]
        close(y, K.scan(*args), K.scan_bound(*args), "y")


@pytest.mark.parametrize("d", [64, 33])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_scan_nonfinite_stays_in_its_channel(ssd, d, bad):
    N, at, ch = 700, 300, 17
    t, h0, g = scan_inputs(1, 2, N, d, "f32", True, True, 6)
    dy = dev(g.standard_normal((1, 2, N, d)).astype(np.float32))
    clean = ssd.gated_scan(*t, scale=2, initial_state=h0)
    grads = ssd.gated_scan_backward(*t, clean, dy, scale=2, initial_state=h0)
    dirty = t[0].clone()
    dirty[0, 1, at, ch] = bad
    y = ssd.gated_scan(dirty, *t[1:], scale=2, initial_state=h0)
    assert not torch.isfinite(y[0, 1, at:, ch]).any()
    y[0, 1, at:, ch] = clean[0, 1, at:, ch]
    assert torch.equal(y, clean)
    dyd = dy.clone()
    dyd[0, 1, at, ch] = bad
    for a, b in zip(ssd.gated_scan_backward(*t, clean, dyd, scale=2, initial_state=h0), grads):
        if a.dim() == 3:
            assert not torch.isfinite(a[0, 1, ch])
            a[0, 1, ch] = b[0, 1, ch]
        else:
            assert not torch.isfinite(a[0, 1, :at + 1, ch]).any()
            a[0, 1, :at + 1, ch] = b[0, 1, :at + 1, ch]
        assert torch.equal(a, b)


@pytest.mark.parametrize("d", [64, 5])
def test_scan_wide_logits(ssd, d):
    """Logits over all of the range that is not counted as infinite, and beyond."""
    g = np.random.default_rng(12)
    shape = (1, 2, 400, d)
    logits = g.uniform(-85, 85, size=(2,) + shape)
    t = [dev(g.standard_normal(shape)), dev(logits[0]), dev(logits[1])]
    dy = dev(g.standard_normal(shape))
    for scale in SCALES:
        args = [f64(v) for v in t] + [None]
        y = ssd.gated_scan(*t, scale=scale)
        close(y, K.scan(*args, scale), K.scan_bound(*args, scale), "y")
        got = ssd.gated_scan_backward(*t, y, dy, scale=scale)
        args += [f64(y), f64(dy), None, scale]
        for name, v, want, bound in zip(("dx", "dA", "dI"), got, K.scan_backward(*args), K.scan_backward_bound(*args)):
            close(v, want, bound, name)
    far = [t[0], t[1].sign() * 1e4, t[2].sign() * 1e4]
    end = [t[0], t[1].sign() * float("inf"), t[2].sign() * float("inf")]
    for scale in SCALES:
        y = ssd.gated_scan(*far, scale=scale)
        assert torch.equal(y, ssd.gated_scan(*end, scale=scale))
        for a, b in zip(ssd.gated_scan_backward(*far, y, dy, scale=scale)[:3],
                        ssd.gated_scan_backward(*end, y, dy, scale=scale)[:3]):
            assert torch.equal(a, b) and bool(torch.isfinite(a).all())


def test_padded_batch(ssd):
    """Padding behind each sequence: logits of -inf keep the last state, and no gradient enters it."""
    g = np.random.default_rng(13)
    B, H, N, d, lengths = 3, 2, 700, 64, (700, 301, 1)
    x, A, dl = g.standard_normal((B, H, N, d)), g.standard_normal((B, H, N, d)) - 3, g.standard_normal((B, H, d))
    for b, n in enumerate(lengths):
        A[b, :, n:] = -np.inf
    t, dl = [dev(x, "bf16"), dev(A, "bf16"), None], dev(dl)
    last = torch.empty((B, H, d), device="cuda")
    y = ssd.gated_scan(*t, scale=2, final_state=last)
    grads = ssd.gated_scan_backward(*t, y, torch.zeros_like(y), scale=2, d_final_state=dl)
    for b, n in enumerate(lengths):
        alone = [v[b:b + 1, :, :n].contiguous() for v in t[:2]] + [None]
        one = torch.empty((1, H, d), device="cuda")
        y1 = ssd.gated_scan(*alone, scale=2, final_state=one)
        # the same sums, in other shares of the workgroups: a few roundings of the state
        assert float((last[b] - one[0]).abs().max()) <= 100 * K.U * float(y1.abs().max() + 1)
        assert torch.equal(last[b], y[b, :, -1])
        g1 = ssd.gated_scan_backward(*alone, y1, torch.zeros_like(y1), scale=2, d_final_state=dl[b:b + 1])
        for a, c in zip(grads[:2], g1[:2]):
            assert bool((a[b, :, n:] == 0).all())
            # lam after n steps: 9 roundings a step (the oracle's STEP) and the joins
            assert float((a[b, :, :n] - c[0]).abs().max()) <= (9 * n + 200) * K.U * float(c.abs().max())


def test_scan_empty(ssd):
    for B, H, N in ((0, 2, 5), (2, 0, 5), (2, 3, 0)):
        x = torch.zeros((B, H, N, 8), device="cuda")
        h0, last = torch.randn((B, H, 8), device="cuda"), torch.full((B, H, 8), 5.0, device="cuda")
        assert ssd.gated_scan(x, x, x, scale=1, initial_state=h0, final_state=last).shape == x.shape
        assert torch.equal(last, h0)
        ssd.gated_scan(x, x, scale=1, final_state=last)
        assert bool((last == 0).all())
        dx, dA, dI, dh0 = ssd.gated_scan_backward(x, x, None, x, x, scale=0, initial_state=h0, d_final_state=h0)
        assert torch.equal(dh0, h0) and dI is None and dx.shape == x.shape
        assert bool((ssd.gated_scan_backward(x, x, None, x, x, scale=0, initial_state=h0)[3] == 0).all())
    none = torch.zeros((0, 3, 8), device="cuda")
    assert ssd.gated_scan_step(none, none, None, none, scale=0).numel() == 0


@pytest.mark.parametrize("S,H,d,dtype,gate", [(1, 1, 1, "f32", False), (3, 2, 33, "bf16", True), (1, 2, 32, "f32", True),
                                              (256, 32, 64, "bf16", True), (7, 5, 128, "bf16", False)])
def test_step(ssd, S, H, d, dtype, gate):
    for scale in SCALES:
        t, h0, _ = scan_inputs(S, H, 1, d, dtype, gate, True, 7, packed=True)
        t = [None if v is None else v[:, :, 0].contiguous() for v in t]
        out = Guard()
        new = ssd.gated_scan_step(*t, h0, scale=scale, new_state=out.empty((S, H, d)))
        args = [None if v is None else f64(v)[:, :, None] for v in t] + [f64(h0), scale]
        close(new[:, :, None], K.scan(*args), K.scan_bound(*args), "step")
        out.check()
        assert ssd.gated_scan_step(*t, h0, scale=scale) is h0  # in place
        assert torch.equal(h0, new)


def test_scan_then_steps(ssd):
    """A prefill's final state, then single tokens, against the whole sequence."""
    B, H, N, d = 3, 4, 200, 64
    t, h0, _ = scan_inputs(B, H, N, d, "bf16", True, True, 8)
    args = [f64(v) for v in t] + [f64(h0), 2]
    want, bound = K.scan(*args), K.scan_bound(*args)
    cut = [v[:, :, :190].contiguous() for v in t]
    state = torch.empty((B, H, d), device="cuda")
    ssd.gated_scan(*cut, scale=2, initial_state=h0, final_state=state)
    for n in range(190, N):
        state = ssd.gated_scan_step(*[v[:, :, n].contiguous() for v in t], state, scale=2)
        close(state, want[:, :, n], bound[:, :, n], f"token {n}")


def test_scan_segments(ssd):
    """A sequence in two calls, the state and its gradient handed over."""
    B, H, N, d, cut = 2, 2, 900, 64, 333
    t, h0, g = scan_inputs(B, H, N, d, "f32", True, True, 9)
    dy, dl = dev(g.standard_normal((B, H, N, d)).astype(np.float32)), dev(g.standard_normal((B, H, d)).astype(np.float32))
    args = [f64(v) for v in t] + [f64(h0)]
    part = [[v[:, :, a:b].contiguous() for v in t] for a, b in ((0, cut), (cut, N))]
    mid = torch.empty((B, H, d), device="cuda")
    y1 = ssd.gated_scan(*part[0], scale=2, initial_state=h0, final_state=mid)
    y2 = ssd.gated_scan(*part[1], scale=2, initial_state=mid)
    y = torch.cat((y1, y2), 2)
    close(y, K.scan(*args, 2), K.scan_bound(*args, 2), "y")
    g2 = ssd.gated_scan_backward(*part[1], y2, dy[:, :, cut:].contiguous(), scale=2, initial_state=mid, d_final_state=dl)
    g1 = ssd.gated_scan_backward(*part[0], y1, dy[:, :, :cut].contiguous(), scale=2, initial_state=h0,
                                 d_final_state=g2[3])
    args += [f64(y), f64(dy), f64(dl), 2]
    want, bound = K.scan_backward(*args), K.scan_backward_bound(*args)
    for i, name in enumerate(("dx", "dA", "dI")):
        close(torch.cat((g1[i], g2[i]), 2), want[i], bound[i], name)
    close(g1[3], want[3], bound[3], "dh0")


# ---- norms ----


def norm_in_inputs(R, E, dtype, seed):
    g = np.random.default_rng(seed)
    r = dev((2 * g.standard_normal((R, E))).astype(np.float32))
    p, du = dev(g.standard_normal((R, E)), dtype), dev(g.standard_normal((R, E)), dtype)
    s, w = (dev((1 + 0.3 * g.standard_normal(E)).astype(np.float32)) for _ in range(2))
    return r, p, s, w, du, dev(g.standard_normal((R, E)).astype(np.float32))


NORM_IN = [(1, 1, "f32"), (3, 7, "bf16"), (5, 64, "f32"), (70, 33, "bf16"), (9, 512, "bf16"), (4, 1000, "f32"),
           (33, 1024, "bf16"), (2, 1025, "bf16"), (6, 2048, "bf16"), (300, 260, "f32"), (3, 4096, "f32"),
           (2, 5001, "bf16"), (2, 16384, "bf16"), (1, 20000, "f32"), (2, 32768, "bf16"), (1, 32767, "f32"),
           (2500, 64, "bf16"), (5000, 36, "f32"),
           (7, 5, "f32"), (7, 6, "bf16"), (40, 129, "f32"), (3, 9001, "bf16"), (2, 2, "bf16"), (1100, 8200, "f32")]


@pytest.mark.parametrize("R,E,dtype", NORM_IN)
@pytest.mark.parametrize("kind", ["scaled", "added", "alone"])
def test_norm_in(ssd, R, E, dtype, kind):
    r, p, s, w, _, _ = norm_in_inputs(R, E, dtype, 1)
    p, s = (p if kind != "alone" else None), (s if kind == "scaled" else None)
    say("norm in", R, E, dtype, kind)
    out = Guard()
    ro = out.empty((R, E)) if p is not None else None
    u = out.empty((R, E), torch_type(dtype))
    got = ssd.norm_in(r, p, s, w, EPS, dtype=torch_type(dtype), residual_out=ro, out=u)
    torch.cuda.synchronize()
    out.check()
    assert got[1] is u and (got[0] is (r if p is None else ro))
    args = [f64(v) for v in (r, p, s, w)] + [EPS]
    for name, v, want, bound in zip(("r", "u"), got, K.norm_in(*args), K.norm_in_bound(*args, dtype)):
        close(v, want, bound, name)


@pytest.mark.parametrize("R,E,dtype", NORM_IN)
@pytest.mark.parametrize("scaled,from_above", [(True, True), (False, True), (True, False)])
def test_norm_in_backward(ssd, R, E, dtype, scaled, from_above):
    r, p, s, w, du, dro = norm_in_inputs(R, E, dtype, 2)
    s = s if scaled else None
    dro = dro if from_above else None
    say("norm in backward", R, E, dtype, scaled, from_above)
    out = Guard()
    dr, dw = out.empty((R, E)), out.empty((E,))
    dp, ds = (out.empty((R, E)), out.empty((E,))) if scaled else (None, None)
    need = ssd.lib().ssd_norm_in_backward_workspace_size(R, E)
    ptr = ssd._ptr
    ws = garbage(need)
    ssd._check(ssd.lib().ssd_norm_in_backward(
        ptr(du), ptr(dro), ptr(r), ptr(p if scaled else None), ptr(s), ptr(w), R, E, EPS, 1 if dtype == "bf16" else 0,
        ptr(dr), ptr(dp), ptr(dw), ptr(ds), ptr(ws), need, ssd._stream(r.device)))
    torch.cuda.synchronize()
    out.check()
    args = [f64(v) for v in (du, dro, r, p, s, w)] + [EPS]
    for name, v, want, bound in zip(("dr", "dp", "dw", "ds"), (dr, dp, dw, ds), K.norm_in_backward(*args),
                                    K.norm_in_backward_bound(*args)):
        if v is not None:
            close(v, want, bound, name)
    again = ssd.norm_in_backward(du, dro, r, p, s, w, EPS)
    assert torch.equal(again[0], dr) and torch.equal(again[2], dw)
    assert again[1] is again[0] if not scaled else torch.equal(again[1], dp) and torch.equal(again[3], ds)


NORM_OUT = [(1, 1, 1, 1, 1, "f32"), (2, 3, 5, 7, 1, "bf16"), (2, 3, 5, 7, 3, "f32"), (1, 2, 70, 32, 1, "bf16"),
            (3, 2, 11, 64, 2, "bf16"), (1, 16, 33, 64, 1, "bf16"), (1, 16, 33, 64, 16, "f32"), (2, 32, 3, 64, 4, "bf16"),
            (5, 32, 1, 64, 1, "bf16"), (1, 12, 9, 33, 1, "bf16"), (1, 64, 2, 128, 1, "f32"), (2, 20, 3, 36, 5, "bf16"),
            (1, 1, 700, 64, 1, "bf16"), (1, 512, 2, 64, 1, "bf16"), (1, 7, 2, 4681, 1, "f32"), (130, 2, 20, 32, 2, "f32"),
            (1, 1, 3000, 4, 1, "bf16"), (2, 600, 2, 64, 2, "f32"),
            (2, 9, 7, 5, 1, "bf16"), (2, 9, 7, 6, 9, "f32"), (3, 8, 40, 33, 2, "bf16"), (2, 5, 3, 3, 1, "bf16"), (1, 500, 3, 2, 1, "f32"),
            (1, 6553, 1, 5, 1, "bf16"), (2, 8, 9, 128, 8, "bf16"), (1, 64, 2, 127, 2, "f32"), (2, 300, 5, 63, 2, "bf16"), (1, 1200, 3, 3, 2, "bf16")]


def norm_out_inputs(B, H, N, d, dtype, seed):
    g = np.random.default_rng(seed)
    y = dev(g.standard_normal((B, H, N, d)).astype(np.float32))
    z, do = (dev(2 * g.standard_normal((B, N, H * d)), dtype) for _ in range(2))
    return y, z, dev((1 + 0.3 * g.standard_normal(H * d)).astype(np.float32)), do


@pytest.mark.parametrize("B,H,N,d,groups,dtype", NORM_OUT)
@pytest.mark.parametrize("first", [True, False])
def test_norm_out(ssd, B, H, N, d, groups, dtype, first):
    y, z, w, _ = norm_out_inputs(B, H, N, d, dtype, 3)
    say("norm out", B, H, N, d, groups, dtype, first)
    out = Guard()
    o = out.empty((B, N, H * d), torch_type(dtype))
    assert ssd.norm_out(y, z, w, EPS, groups=groups, gate_first=first, out=o) is o
    torch.cuda.synchronize()
    out.check()
    args = [f64(v) for v in (y, z, w)] + [groups, first, EPS]
    close(o, K.norm_out(*args), K.norm_out_bound(*args, dtype), "o")


@pytest.mark.parametrize("B,H,N,d,groups,dtype", NORM_OUT)
@pytest.mark.parametrize("first", [True, False])
def test_norm_out_backward(ssd, B, H, N, d, groups, dtype, first):
    y, z, w, do = norm_out_inputs(B, H, N, d, dtype, 4)
    say("norm out backward", B, H, N, d, groups, dtype, first)
    out = Guard()
    dy, dz, dw = out.empty(y.shape), out.empty(z.shape), out.empty(w.shape)
    need = ssd.lib().ssd_norm_out_backward_workspace_size(B, H, N, d, groups)
    ptr = ssd._ptr
    ws = garbage(need)
    ssd._check(ssd.lib().ssd_norm_out_backward(
        ptr(do), ptr(y), ptr(z), ptr(w), B, H, N, d, groups, 1 if first else 0, EPS, 1 if dtype == "bf16" else 0,
        ptr(dy), ptr(dz), ptr(dw), ptr(ws), need, ssd._stream(y.device)))
    torch.cuda.synchronize()
    out.check()
    args = [f64(v) for v in (do, y, z, w)] + [groups, first, EPS]
    got = (dy, dz, dw)
    for name, v, want, bound in zip(("dy", "dz", "dw"), got, K.norm_out_backward(*args),
                                    K.norm_out_backward_bound(*args)):
        close(v, want, bound, name)
    for a, b in zip(got, ssd.norm_out_backward(do, y, z, w, EPS, groups=groups, gate_first=first)):
        assert torch.equal(a, b)


def test_norm_rows_of_zeros_and_infinities(ssd):
    """A row of zeros gives zeros with eps > 0 and NaN with eps = 0; a row with an
    infinity gives NaN there and 0 beside it; other rows are untouched."""
    E = 64
    r, _, _, w, _, _ = norm_in_inputs(4, E, "f32", 5)
    clean = ssd.norm_in(r, None, None, w, EPS, dtype=torch.float32)[1]
    r[1] = 0
    r[2, 5] = float("inf")
    u = ssd.norm_in(r, None, None, w, EPS, dtype=torch.float32)[1]
    assert bool((u[1] == 0).all()) and bool(torch.isnan(u[2, 5])) and int(torch.isnan(u[2]).sum()) == 1
    assert bool((u[2, :5] == 0).all()) and torch.equal(u[0], clean[0]) and torch.equal(u[3], clean[3])
    assert bool(torch.isnan(ssd.norm_in(r, None, None, w, 0.0, dtype=torch.float32)[1][1]).all())
    y, z, w, _ = norm_out_inputs(1, 2, 3, 32, "f32", 6)
    z[0, 1] = -1e4  # a gate shut all along the row
    for first in (True, False):
        o = ssd.norm_out(y, z, w, EPS, gate_first=first)
        assert bool((o[0, 1] == 0).all()) and bool(torch.isfinite(o).all())


def test_norm_empty(ssd):
    w = torch.ones(8, device="cuda")
    x = torch.empty((0, 8), device="cuda")
    assert ssd.norm_in(x, x, w, w, EPS)[1].shape == (0, 8)
    dr, dp, dw, ds = ssd.norm_in_backward(x, x, x, x, w, w, EPS)
    assert bool((dw == 0).all()) and bool((ds == 0).all())
    y = torch.empty((2, 2, 0, 4), device="cuda")
    z = torch.empty((2, 0, 8), device="cuda")
    assert ssd.norm_out(y, z, w, EPS).shape == z.shape
    assert bool((ssd.norm_out_backward(z, y, z, w, EPS)[2] == 0).all())


# ---- together ----


def block(ssd, P, r, branch, mixer):
    """One block as a model runs it: the residual stream and the previous block's
    branch in, the residual stream and this block's branch out."""
    B, N, E = r.shape
    H, d = P["H"], E // P["H"]
    r, u = ssd.norm_in(r, branch, P["s"], P["w_in"], EPS)
    heads = lambda m: (u.float() @ m).view(B, N, H, d).transpose(1, 2).contiguous().to(branch.dtype)  # noqa: E731
    z = (u.float() @ P["Wz"]).to(branch.dtype)
    y = mixer(*[heads(m) for m in P["W"]])
    o = ssd.norm_out(y, z, P["w_out"], EPS, groups=P["groups"])
    return r, (o.float() @ P["Wo"]).to(branch.dtype)


def block_params(E, H, groups, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return dict(H=H, groups=groups, s=0.5 + 0.1 * n(E), w_in=1 + 0.1 * n(E), w_out=1 + 0.1 * n(E),
                W=[n(E, E) / E ** 0.5 for _ in range(3)], Wz=n(E, E) / E ** 0.5, Wo=n(E, E) / E ** 0.5)


def test_blocks_with_both_mixers(ssd):
    """A gated-recurrence block and an order-1 mixer block behind it; the same
    tokens one at a time through the recurrence block give the same outputs."""
    B, N, E, H = 2, 150, 256, 4
    g = torch.Generator(device="cuda").manual_seed(3)
    r0 = torch.randn((B, N, E), generator=g, device="cuda")
    b0 = torch.randn((B, N, E), generator=g, device="cuda")
    P, Q = block_params(E, H, 1, 1), block_params(E, H, H, 2)
    rec = lambda x, A, I: ssd.gated_scan(x, A, I, scale=2)  # noqa: E731
    r1, b1 = block(ssd, P, r0, b0, rec)

    def ssm(q, k, v):
        dt, a_cs, _ = ssd.prep_amask(v[..., 0].contiguous() - 3, None, 64)
        return ssd.forward(q.abs() + 0.1, k.abs() + 0.1, v, None, a_cs, 1, 64)

    r2, b2 = block(ssd, Q, r1, b1, ssm)
    assert bool(torch.isfinite(r2).all()) and bool(torch.isfinite(b2).all())
    state = torch.zeros((B, H, E // H), device="cuda")

    def one(x, A, I):
        ssd.gated_scan_step(x[:, :, 0].contiguous(), A[:, :, 0].contiguous(), I[:, :, 0].contiguous(), state, scale=2)
        return state.view(B, H, 1, E // H)

    for n in range(N):
        rn, bn = block(ssd, P, r0[:, n:n + 1].contiguous(), b0[:, n:n + 1].contiguous(), one)
        assert torch.equal(rn[:, 0], r1[:, n])
        # the projections' sums are taken in another order for one token: 256 terms, 1e-5 of the row
        err = (bn[:, 0] - b1[:, n]).norm() / b1[:, n].norm()
        assert float(err) < 1e-4, (n, float(err))


def test_chain_gradients(ssd):
    """norm_in -> gated_scan -> norm_out backwards, against torch's differentiation
    of the same chain in 64 bits."""
    B, N, H, d = 2, 90, 3, 32
    E = H * d
    g = torch.Generator(device="cuda").manual_seed(4)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    r, p, z, do, dr_out = n(B, N, E), n(B, N, E), n(B, N, E), n(B, N, E), n(B, N, E)
    s, w1, w2 = 1 + 0.1 * n(E), 1 + 0.1 * n(E), 1 + 0.1 * n(E)
    A, I = n(B, H, N, d) - 2, n(B, H, N, d)
    r2, u = ssd.norm_in(r, p, s, w1, EPS)
    x = u.view(B, N, H, d).transpose(1, 2).contiguous()
    y = ssd.gated_scan(x, A, I, scale=2)
    dy, dz, dw2 = ssd.norm_out_backward(do, y, z, w2, EPS)
    dx, dA, dI, _ = ssd.gated_scan_backward(x, A, I, y, dy, scale=2)
    du = dx.transpose(1, 2).reshape(B, N, E)
    dr, dp, dw1, ds = ssd.norm_in_backward(du, dr_out, r2, p, s, w1, EPS)
    got = dict(r=dr, p=dp, s=ds, w1=dw1, A=dA, I=dI, z=dz, w2=dw2)
    v = {k: t.double().cpu().requires_grad_() for k, t in dict(r=r, p=p, s=s, w1=w1, A=A, I=I, z=z, w2=w2).items()}
    R = v["r"] + v["s"] * v["p"]
    U = R / (R.square().mean(-1, keepdim=True) + EPS).sqrt() * v["w1"]
    X = U.view(B, N, H, d).transpose(1, 2)
    a = torch.sigmoid(-v["A"])
    src = torch.sqrt(1 - a * a) * torch.sigmoid(v["I"]) * X
    h, hs = torch.zeros((B, H, d), dtype=torch.float64), []
    for t in range(N):
        h = a[:, :, t] * h + src[:, :, t]
        hs.append(h)
    T = torch.stack(hs, 2).transpose(1, 2).reshape(B, N, E) * torch.nn.functional.silu(v["z"])
    O = T / (T.square().mean(-1, keepdim=True) + EPS).sqrt() * v["w2"]
    (R * dr_out.double().cpu()).sum().add((O * do.double().cpu()).sum()).backward()
    for k, t in got.items():
        want = v[k].grad
        err = float((t.double().cpu() - want).norm() / want.norm())
        say(f"  {k}: {err:.3g}")
        # three operators of at most a few hundred fp32 roundings each, 300 * 2^-24 a piece
        assert err < 6e-5, (k, err)


def every_call(ssd, seed):
    """One call of every operator: (name, function)."""
    t, h0, g = scan_inputs(2, 4, 1300, 64, "bf16", True, True, seed)
    y = ssd.gated_scan(*t, scale=2, initial_state=h0)
    dy, dl = torch.randn_like(y), torch.randn_like(h0)
    s = [v[:, :, 0].contiguous() for v in t]
    r, p, sc, w, du, dro = norm_in_inputs(300, 1024, "bf16", seed)
    yo, z, wo, do = norm_out_inputs(2, 16, 100, 64, "bf16", seed)
    return [
        ("scan", lambda: (ssd.gated_scan(*t, scale=2, initial_state=h0),)),
        ("scan backward", lambda: ssd.gated_scan_backward(*t, y, dy, scale=2, initial_state=h0, d_final_state=dl)),
        ("step", lambda: (ssd.gated_scan_step(*s, h0, scale=2, new_state=torch.empty_like(h0)),)),
        ("norm in", lambda: ssd.norm_in(r, p, sc, w, EPS)),
        ("norm in backward", lambda: ssd.norm_in_backward(du, dro, r, p, sc, w, EPS)),
        ("norm out", lambda: (ssd.norm_out(yo, z, wo, EPS),)),
        ("norm out backward", lambda: ssd.norm_out_backward(do, yo, z, wo, EPS)),
    ]


def test_refused_on_the_gpu(ssd):
    """What the binding refuses of GPU tensors: types, shapes, strides, one operand on the host."""
    x = torch.randn((1, 2, 8, 4), device="cuda")
    h = torch.zeros((1, 2, 4), device="cuda")
    w, rows = torch.ones(4, device="cuda"), torch.randn((6, 4), device="cuda")
    wide = torch.randn((1, 2, 8, 8), device="cuda")[..., ::2]
    bad = [
        lambda: ssd.gated_scan(x, x.bfloat16(), scale=0),
        lambda: ssd.gated_scan(x.half(), x.half(), scale=0),
        lambda: ssd.gated_scan(x, x[:, :, :4].contiguous(), scale=0),
        lambda: ssd.gated_scan(wide, x, scale=0),
        lambda: ssd.gated_scan(x, wide, scale=0),
        lambda: ssd.gated_scan(x, x.cpu(), scale=0),
        lambda: ssd.gated_scan(x, x, scale=0, initial_state=x),
        lambda: ssd.gated_scan(x, x, scale=0, y=x.bfloat16()),
        lambda: ssd.gated_scan_step(x[:, :, 0].contiguous(), x[:, :, 1].contiguous(), None, h.cpu(), scale=0),
        lambda: ssd.gated_scan_backward(x, x, None, x.bfloat16(), x, scale=0),
        lambda: ssd.norm_in(rows.bfloat16(), rows, None, w, EPS),
        lambda: ssd.norm_in(rows, rows[:5], None, w, EPS),
        lambda: ssd.norm_in(rows, rows, w[:3], w, EPS),
        lambda: ssd.norm_in(rows, rows, None, w, EPS, out=rows.bfloat16()),
        lambda: ssd.norm_in_backward(rows, None, rows, None, w, w, EPS),
        lambda: ssd.norm_in_backward(rows, None, rows.cpu(), None, None, w, EPS),
        lambda: ssd.norm_out(x, rows, w, EPS),
        lambda: ssd.norm_out(x, torch.randn((1, 8, 8), device="cuda"), w, EPS),
        lambda: ssd.norm_out_backward(rows, x, torch.randn((1, 8, 8), device="cuda"), torch.ones(8, device="cuda"), EPS),
    ]
    for k, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print("not refused:", k)
    for f in (lambda: ssd.gated_scan(x, None, scale=0), lambda: ssd.gated_scan(x, x, scale=3),
              lambda: ssd.gated_scan(x, x, scale=0, y=x), lambda: ssd.norm_in(rows, rows, None, w, -1.0),
              lambda: ssd.norm_in(rows, rows, None, w, EPS, residual_out=rows),
              lambda: ssd.gated_scan(x, x, scale=0, initial_state=h, final_state=h),
              lambda: ssd.norm_out(x, torch.randn((1, 8, 8), device="cuda"), torch.ones(8, device="cuda"), EPS, groups=3)):
        with pytest.raises(ssd.SSDError):
            f()
    for f in (lambda: ssd.gated_scan_backward(x, x, None, None, x, scale=0),
              lambda: ssd.norm_in_backward(rows, None, None, None, None, w, EPS),
              lambda: ssd.norm_in(None, rows, None, w, EPS)):
        with pytest.raises(TypeError):
            f()


def test_same_bits_every_time(ssd):
    for name, f in every_call(ssd, 21):
        first = f()
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(first, f())), name


def test_other_streams(ssd):
    """Calls on two streams at once, each with its own workspace."""
    calls = every_call(ssd, 22)
    want = [f() for _, f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _, f in calls:
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(f())
    torch.cuda.synchronize()
    for k in range(2):
        for (name, _), a, b in zip(calls, want, got[k]):
            assert all(torch.equal(u, v) for u, v in zip(a, b)), name


def test_captured(ssd):
    """Every call in one captured graph, replayed on new inputs between eager calls."""
    calls = every_call(ssd, 23)
    x = torch.randn((1, 2, 700, 64), device="cuda")
    A, dy = torch.randn_like(x) - 3, torch.randn_like(x)

    def chain():
        y = ssd.gated_scan(x, A, A, scale=1)
        return (y,) + ssd.gated_scan_backward(x, A, A, y, dy, scale=1)[:3]

    for _, f in calls:
        f()
    chain()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [f() for _, f in calls]
        linked = chain()
    for k in range(4):
        x.normal_()
        A.normal_()
        graph.replay()
        want = [f() for _, f in calls]
        again = chain()
        torch.cuda.synchronize()
        for (name, _), a, b in zip(calls, got, want):
            assert all(torch.equal(u, v) for u, v in zip(a, b)), (k, name)
        assert all(torch.equal(u, v) for u, v in zip(linked, again)), k


def test_offsets_past_2e31_elements(ssd):
    """2.28e9 elements an array: every copy of the first heads (rows) gives their bits."""
    N, d, copies = 65536, 64, 68
    g = torch.Generator(device="cuda").manual_seed(1)
    one = [torch.randn((1, 8, N, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    one[1] -= 3
    small = ssd.gated_scan(*one, scale=2)
    big = [v.expand(copies, 8, N, d).contiguous() for v in one]
    y = ssd.gated_scan(*big, scale=2)
    # the work may be split otherwise for more heads: within the roundings of the joins
    err = (y[0] - small[0]).abs().max() / small.abs().max()
    assert float(err) < 1e-5
    for c in range(1, copies):
        assert torch.equal(y[c], y[0]), c
    say("scan done")
    del big
    w = torch.ones(8 * d, device="cuda")
    z = one[0].view(1, N, 8 * d).expand(copies, N, 8 * d).contiguous()
    o = ssd.norm_out(y, z, w, EPS)
    for c in range(1, copies):
        assert torch.equal(o[c], o[0]), c
    assert torch.equal(o[0], ssd.norm_out(y[:1].contiguous(), z[:1].contiguous(), w, EPS)[0])
    say("norm out done")
    rows = y.view(copies * N, 8 * d)
    r2, u = ssd.norm_in(rows, o.view(copies * N, 8 * d), None, w, EPS)
    first = r2[:N].clone(), u[:N].clone()
    for c in range(1, copies):
        assert torch.equal(r2[c * N:(c + 1) * N], first[0]) and torch.equal(u[c * N:(c + 1) * N], first[1]), c


def test_backward_offsets_past_2e31_elements(ssd):
    N, d, copies = 65536, 64, 68
    g = torch.Generator(device="cuda").manual_seed(2)
    x, A = (torch.randn((1, 8, N, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    y = ssd.gated_scan(x, A, scale=1)
    big = [v.expand(copies, 8, N, d).contiguous() for v in (x, A, y, y)]
    dx, dA, _, _ = ssd.gated_scan_backward(big[0], big[1], None, big[2], big[3], scale=1)
    for c in range(1, copies):
        assert torch.equal(dx[c], dx[0]) and torch.equal(dA[c], dA[0]), c
    small = ssd.gated_scan_backward(x, A, None, y, y, scale=1)
    assert float((dx[0] - small[0][0]).abs().max() / dx[0].abs().max()) < 1e-5
    say("scan backward done")
    del dx, dA, small
    w = torch.ones(8 * d, device="cuda")
    z = big[0].view(copies, N, 8 * d)
    dy, dz, dw = ssd.norm_out_backward(z, big[2], z, w, EPS)
    for c in range(1, copies):
        assert torch.equal(dy[c], dy[0]) and torch.equal(dz[c], dz[0]), c
    assert bool(torch.isfinite(dw).all())
    del dy, dz
    rows = big[2].view(copies * N, 8 * d)
    dr, _, dw, _ = ssd.norm_in_backward(z.view(copies * N, 8 * d), rows, rows, None, None, w, EPS)
    first = dr[:N].clone()
    for c in range(1, copies):
        assert torch.equal(dr[c * N:(c + 1) * N], first), c
    assert bool(torch.isfinite(dw).all())
