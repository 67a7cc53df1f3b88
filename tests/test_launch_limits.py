"""Calls whose grid a launch cannot hold (2^32 threads and more, which HIP starts
only in part, without an error) are refused before any HIP call; calls that just
fit are taken.  Fake, never dereferenced addresses; what is taken is stopped by a
misaligned pointer, a missing workspace or a missing array before its launch."""
import pytest

from mamba_ssd_sequence_amd import ssd as binding

P = [i << 48 for i in range(1, 30)]  # 256 TB apart
ODD = P[20] + 4


@pytest.fixture(scope="module")
def lib():
    return binding.lib()


def refused(lib, status):
    return status == 2 and any(w in lib.ssd_last_error().decode() for w in ("grid", "state too large", "H too large"))


# A chunk of 64 has a wave of 64 lanes, or 16 lanes of one where N is a multiple of 4.
@pytest.mark.parametrize("BH,N,chunk", [(1 << 26, 1, 64), (1 << 25, 65, 64), (1 << 28, 4, 64), (1 << 26, 1, 128),
                                        (1 << 27, 4, 128)])
def test_prep(lib, BH, N, chunk):
    prep = lambda BH, last: lib.ssd_prep(P[0], P[1], P[2], BH, 1, N, chunk, P[3], P[4], last, None)  # noqa: E731
    amask = lambda BH, last: lib.ssd_prep_amask(P[0], P[1], BH, 1, N, chunk, P[3], P[4], last, None)  # noqa: E731
    for call in (prep, amask):
        assert refused(lib, call(BH, P[5]))
        assert call(BH - 64, ODD) == 4


@pytest.mark.parametrize("order,dtype,d,N,init,BH", [
    (1, 1, 32, 1, False, 1 << 24),                       # the scan: a workgroup of 256 a head
    (1, 0, 32, 1, False, -(-(1 << 24) // 5)),            # 1056 values of a state: 5 workgroups a head
    (1, 0, 64, 1, True, -(-(1 << 24) // 17)),            # 4160: 17
    (1, 0, 64, 64 * 40, False, -(-(1 << 24) // 40)),     # 40 blocks
    (2, 1, 64, 1, False, 1 << 20),                       # 8 workgroups of 512 a head
    (2, 1, 64, 1, True, 1 << 18),                        # 64 of 256 for the initial state
    (2, 1, 64, 64 * 40, False, (1 << 24) // 40 + 8)])    # 40 blocks
def test_forward(lib, order, dtype, d, N, init, BH):
    def call(BH):
        return lib.ssd_forward(P[0], P[1], P[2], P[3], P[4], P[5] if init else None, P[6] if init else None, BH, 1, N, d,
                               order, 64, dtype, P[7], None, None, None, None, 0, None)

    assert refused(lib, call(BH))
    assert call(BH - 17) == 6


def test_forward_scan_of_many_blocks(lib):
    """The scan's grid does not grow with the blocks: 2^24 of them in 2^23 heads are taken."""
    assert lib.ssd_forward(P[0], P[1], P[2], P[3], P[4], None, None, 1 << 23, 1, 65, 32, 1, 64, 1, P[7], None, None, None,
                           None, 0, None) == 6


@pytest.mark.parametrize("order,dtype,d,N,BH", [
    (1, 0, 32, 1, -(-(1 << 24) // 5)), (1, 1, 64, 1, -(-(1 << 24) // 17)), (1, 1, 64, 64 * 40, -(-(1 << 24) // 40)),
    (2, 1, 64, 1, 1 << 18), (2, 1, 64, 64 * 100, -(-(1 << 24) // 100))])
def test_backward(lib, order, dtype, d, N, BH):
    def call(BH):
        return lib.ssd_backward(P[0], P[1], P[2], P[3], P[4], P[5], P[6], P[7], BH, 1, N, d, order, 64, dtype, P[8], P[9],
                                P[10], P[11], P[12], None, 0, None)

    assert refused(lib, call(BH))
    assert call(BH - 1) == 6


@pytest.mark.parametrize("order,d,layout,S", [(1, 32, 0, 1 << 24), (2, 32, 0, 1 << 22), (2, 64, 1, 1 << 23)])
def test_decode(lib, order, d, layout, S):
    def call(S, y):
        return lib.ssd_decode_step(P[0], P[1], P[2], P[3], P[4], P[5], S, 1, d, order, 1, layout, P[6], P[7], y, None)

    assert refused(lib, call(S, P[8]))
    assert call(S - 1, ODD) == 4


def test_state_layout(lib):
    for call in (lib.ssd_state_pack, lib.ssd_state_unpack):
        for d in (32, 64):
            BH = (1 << 24) // d
            assert refused(lib, call(P[0], P[1], BH, d, P[2], P[3], None))
            assert call(P[0], P[1], BH - 1, d, ODD, P[3], None) == 4


def test_prep_backward(lib):
    def call(H, last):
        return lib.ssd_prep_backward(P[0], P[1], P[2], P[3], None, 1, H, 1, P[4], P[5], last, None)

    def amask(H, last):
        return lib.ssd_prep_amask_backward(P[0], None, P[1], None, 1, H, 1, last, None, None)

    for f in (call, amask):
        assert refused(lib, f(1 << 22, P[6]))
        assert f((1 << 22) - 1, ODD) == 4
