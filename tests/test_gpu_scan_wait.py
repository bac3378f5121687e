"""A scan one of whose waits runs out: every block of its cluster unwinds, the status says so,
and the next calls are right.  The failure is a tile that the kernel is told not to fetch."""
import time

import pytest
import torch

from linear_attention_12_b200 import gdn

BF16, F32 = torch.bfloat16, torch.float32


def test_refusals():
    with pytest.raises(TypeError):
        gdn.selftest_scan_wait(torch.zeros(5, 8, 64), 0)
    L = gdn.lib()
    P = 0x10000  # never dereferenced: refused on the host
    for T, C, tile, p in ((8, 64, -1, P), (0, 64, 0, P), (8, 0, 0, P), (8, 64, 0, None),
                          (8, 64, 0, P + 2)):
        assert L.gdn_selftest_scan_wait(0, p, T, C, tile, None) == gdn.GDN_ERR_INVALID_ARG


# (tiles of 64 or 128 rows: by TMA and by granules, one and several blocks a cluster; the first
# turn, a turn in the middle, the last tile)
@pytest.mark.gpu
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("T,C,tile", [(50, 64, 0), (700, 64, 0), (9000, 64, 40), (9000, 64, 70),
                                      (9000, 515, 37), (5000, 2048, 0), (5000, 2048, 50),
                                      (5000, 2048, 78), (5000, 2051, 60)])
def test_a_tile_that_never_comes(T, C, tile, backward):
    assert gdn.last_device_error() == gdn.GDN_OK
    g = torch.Generator("cuda").manual_seed(T + C)
    b = torch.randn(5, T, C, generator=g, device="cuda")
    b[0].abs_().neg_()
    h, hf = gdn.scan(b[1], b[0])
    back = gdn.scan_backward(b[0], h, b[1])
    t0 = time.monotonic()
    gdn.selftest_scan_wait(b, tile, backward=backward)
    assert gdn.last_device_error() == gdn.GDN_ERR_TIMEOUT
    assert time.monotonic() - t0 < 2.0  # a few waits of 20 to 40 ms, not one per turn
    assert gdn.last_device_error() == gdn.GDN_OK
    again = (*gdn.scan(b[1], b[0]), *gdn.scan_backward(b[0], h, b[1]))
    assert all(torch.equal(p, q) for p, q in zip(again, (h, hf, *back)))
    assert gdn.last_device_error() == gdn.GDN_OK


@pytest.mark.gpu
def test_no_such_tile():
    """The short limit alone disturbs nothing."""
    g = torch.Generator("cuda").manual_seed(1)
    b = torch.randn(5, 1000, 128, generator=g, device="cuda")
    b[0].abs_().neg_()
    gdn.selftest_scan_wait(b, 1 << 20)
    assert gdn.last_device_error() == gdn.GDN_OK
    assert torch.equal(b[2], gdn.scan(b[1], b[0])[0])
    h, dx, dla = b[1].clone(), b[3], b[4]
    gdn.selftest_scan_wait(b, 1 << 20, backward=True)
    assert gdn.last_device_error() == gdn.GDN_OK
    ref = gdn.scan_backward(b[0], h, b[2])
    assert torch.equal(dx, ref[0]) and torch.equal(dla, ref[1])
