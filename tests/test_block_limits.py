"""Calls at the ends of their sizes: what a launch cannot hold is refused before
any HIP call or taken in several launches."""
import pytest

from mamba_ssd_sequence_amd import ssd as binding
from oracle import block_oracle as K
from test_block_gpu import SCALES, bounded_backward, bounded_scan, close, dev, f64, say, scan_inputs

FAR = [i << 45 for i in range(1, 20)]  # fake addresses 32 TB apart


@pytest.fixture(scope="module")
def lib():
    return binding.lib()


def scan(lib, B, H, N, d, dtype, wsb=0):
    return lib.ssd_gated_scan(FAR[0], FAR[1], FAR[2], None, B, H, N, d, 2, dtype, FAR[3], None, FAR[4], wsb, None)


def scan_back(lib, B, H, N, d, dtype, wsb=0):
    return lib.ssd_gated_scan_backward(FAR[0], FAR[1], None, None, FAR[3], FAR[4], None, B, H, N, d, 2, dtype, FAR[5],
                                       FAR[6], None, None, FAR[7], wsb, None)


# One head's threads: a tile of 8 waves has 128 tokens of 64 channels (256 in bf16
# forwards), so 2^23 tiles of 512 threads are 2^32, one more than a launch holds.
# Without a workspace the largest call that fits is refused for that (6) instead.
@pytest.mark.parametrize("call,dtype,N,d", [(scan, 0, 1 << 30, 64), (scan, 1, 1 << 31, 64), (scan_back, 1, 1 << 30, 64),
                                            (scan, 0, 1 << 28, 256), (scan_back, 0, 1 << 28, 200)])
def test_a_head_larger_than_a_launch(lib, call, dtype, N, d):
    assert call(lib, 1, 1, N, d, dtype) == 2
    assert "grid" in lib.ssd_last_error().decode()
    assert call(lib, 1, 1, N - 256, d, dtype) == 6


def test_steps_larger_than_a_launch(lib):
    step = lambda S, d, out: lib.ssd_gated_scan_step(FAR[0], FAR[1], None, FAR[2], S, 1, d, 0, 1, out, None)  # noqa: E731
    assert step((1 << 30) - 1, 16, FAR[3]) == 2  # 2^34 - 16 channels: 2^24 workgroups of 256 threads
    assert step((1 << 30) - 64, 16, None) == 1   # 2^34 - 1024: taken, but for the missing output


def test_norm_out_larger_than_a_launch(lib):
    def fwd(H, d, o):
        return lib.ssd_norm_out(FAR[0], FAR[1], FAR[2], 1, H, 1, d, H, 1, 1e-5, 1, o, None)

    def back(H, d, dw):
        return lib.ssd_norm_out_backward(FAR[0], FAR[1], FAR[2], FAR[3], 1, H, 1, d, H, 1, 1e-5, 1, FAR[4], FAR[5], dw,
                                         FAR[6], 0, None)

    assert fwd(1 << 28, 1, FAR[3]) == 2 and fwd((1 << 28) - 32, 1, None) == 1
    assert back(1 << 21, 64, FAR[7]) == 2 and back((1 << 21) - 1, 64, None) == 1


@pytest.mark.gpu
def test_more_heads_than_a_launch_holds():
    """2^23 + 3 heads of 512 threads each: two launches, every copy of the first heads with their bits."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    BH, few, N, d = (1 << 23) + 3, 509, 3, 4
    g = torch.Generator(device="cuda").manual_seed(6)

    def heads(*rest):
        one = torch.randn((few,) + rest, generator=g, device="cuda")
        return one.repeat(-(-BH // few), *[1] * len(rest))[:BH].unsqueeze(0).contiguous()

    x, A, I = (heads(N, d).bfloat16() for _ in range(3))
    dy, h0, dl = heads(N, d), heads(d), heads(d)
    last = torch.empty_like(h0)
    y = binding.gated_scan(x, A, I, scale=2, initial_state=h0, final_state=last)
    grads = binding.gated_scan_backward(x, A, I, y, dy, scale=2, initial_state=h0, d_final_state=dl)
    torch.cuda.synchronize()
    assert torch.equal(last, y[:, :, -1])
    f64 = lambda t: t[:, :few].double().cpu().numpy()  # noqa: E731
    args = [f64(t) for t in (x, A, I, h0)]
    back = args + [f64(t) for t in (y, dy, dl)] + [2]
    for name, got, want, bound in zip(("y", "dx", "dA", "dI", "dh0"), (y, *grads),
                                      (K.scan(*args, 2), *K.scan_backward(*back)),
                                      (K.scan_bound(*args, 2), *K.scan_backward_bound(*back))):
        print("heads past a launch", name, flush=True)
        assert (abs(f64(got) - want) <= bound).all(), name
        for a in range(0, BH, few):  # torch's comparisons of whole copies, on the GPU
            b = min(a + few, BH)
            if a % (1 << 12) < few or b > BH - 4 * few:
                assert torch.equal(got[:, a:b], got[:, :b - a]), (name, a)
        whole = got[0, :BH // few * few].view(BH // few, few, -1)
        assert bool((whole == whole[:1]).all()), name


@pytest.mark.gpu
def test_norm_in_refuses_another_type_than_the_branch():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    r, w = torch.randn((3, 64), device="cuda"), torch.ones(64, device="cuda")
    p = torch.randn_like(r).bfloat16()
    want = binding.norm_in(r, p, None, w, 1e-5)[1]
    assert want.dtype == torch.bfloat16
    assert torch.equal(binding.norm_in(r, p, None, w, 1e-5, dtype=torch.bfloat16)[1], want)
    for branch, other in ((p, torch.float32), (r, torch.bfloat16), (p, torch.float16)):
        with pytest.raises(ValueError, match="branch"):
            binding.norm_in(r, branch, None, w, 1e-5, dtype=other)


# From 512 heads (and slabs of 64 channels) on, where they fill the chip's rounds, a
# workgroup takes up to 8 tiles of a head one after the other; else the tiles are
# shared out (833 heads).  600 tokens are 3 tiles of 64 channels, backwards 5.
@pytest.mark.gpu
@pytest.mark.parametrize("B,H,N,d,dtype,gate,init,packed", [
    (64, 8, 600, 64, "bf16", True, True, True), (16, 16, 1000, 80, "bf16", True, False, False),
    (48, 16, 300, 17, "f32", False, True, False), (128, 4, 2100, 3, "bf16", True, True, True),
    (119, 7, 300, 64, "f32", True, True, False)])
def test_scan_of_many_heads(B, H, N, d, dtype, gate, init, packed):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    for scale in SCALES:
        t, h0, g = scan_inputs(B, H, N, d, dtype, gate, init, 14, packed)
        say("scan of many heads", B, H, N, d, dtype, gate, init, packed, scale)
        y, last = bounded_scan(binding, t, h0, scale)
        args = [f64(v) for v in t] + [f64(h0)]
        want, bound = K.scan(*args, scale), K.scan_bound(*args, scale)
        close(y, want, bound, "y")
        assert torch.equal(last, y[:, :, -1])
        dy, dl = dev(g.standard_normal(y.shape)), dev(g.standard_normal(h0.shape)) if init else None
        got = bounded_backward(binding, t, h0, y, dy, dl, scale)
        args += [f64(y), f64(dy), f64(dl), scale]
        for name, v, want, bound in zip(("dx", "dA", "dI", "dh0"), got, K.scan_backward(*args),
                                        K.scan_backward_bound(*args)):
            if v is not None:
                close(v, want, bound, name)
