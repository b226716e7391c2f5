"""Which kernels a product takes, on a card of 256 CUs (CPU): rows stream where a weight's bytes are
the cost, and go through tiles where streaming would walk them pass after pass on a few CUs."""
import pytest

from tests.product_choice import streams


def cross(mode, N, K, G):
    """The largest M that streams."""
    lo, hi = 0, 1 << 27
    while lo < hi:
        mid = (lo + hi + 1) // 2
        lo, hi = (mid, hi) if streams(mode, mid, N, K, G, cus=256) else (lo, mid - 1)
    return lo


@pytest.mark.parametrize("mode", ["w4a16", "w4a4"])
@pytest.mark.parametrize("M,N,K,G", [(512, 16, 4096, 1), (1024, 256, 4096, 1), (1200, 256, 1024, 1),
                                     (700, 512, 4096, 2), (520, 96, 7168, 1)])
def test_many_rows_of_a_narrow_product_go_through_tiles(mode, M, N, K, G):
    """Measured 1.2 to 5.2 times as long when streamed."""
    assert not streams(mode, M, N, K, G, cus=256)


@pytest.mark.parametrize("mode", ["w4a16", "w4a4", "backward"])
def test_few_rows_stream_however_few_outputs(mode):
    for N, K in ((16, 4096), (256, 4096), (4096, 4096), (64, 8224), (65536, 32)):
        for G in (1, 8, 160, 1024):
            m = cross(mode, N, K, G)
            assert 20 * G <= m <= 300 * G, (N, K, G, m)
            assert streams(mode, 1, N, K, G, cus=256)


def test_measured_crossings():
    """Rows at which the two take the same time (64 groups, and one, of 2048 x 4096), within the
    steps measured: streamed at the lower count, tiled at the upper."""
    for mode, G, lower, upper in (("w4a16", 64, 16 * 64, 32 * 64), ("w4a4", 64, 16 * 64, 32 * 64),
                                  ("backward", 64, 32 * 64, 47 * 64), ("w4a16", 1, 128, 384), ("w4a4", 1, 128, 256)):
        assert lower <= cross(mode, 2048, 4096, G) < upper, (mode, G)


def test_rows_out_of_the_tiles_reach_stream():
    for mode in ("w4a16", "backward"):
        assert not streams(mode, 100000, 512, 512, 4, stride=1 << 22, cus=256)
        assert streams(mode, 100000, 512, 512, 4, stride=(1 << 22) + 1, cus=256)
