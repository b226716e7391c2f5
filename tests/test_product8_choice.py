"""Which kernels a product of MXFP8 rows takes, on a card of 256 CUs (CPU): the launches' own rule."""
import ctypes

import pytest

import nvfp4_expert_layer_amd as nv


def streams(M, N, K, G, cus=256):
    f = nv.lib().moe_internal_product_streams
    f.argtypes = [ctypes.c_int] * 4 + [ctypes.c_int64] + [ctypes.c_int] * 3
    f.restype = ctypes.c_int
    return bool(f(M, N, K, G, K, 2, 0, cus))


@pytest.mark.parametrize("G,N,K,lower,upper", [(160, 2048, 4128, 32, 48), (64, 2048, 4128, 32, 48), (8, 2048, 4128, 96, 128),
                                               (16, 1024, 2080, 96, 128), (1, 4096, 4128, 192, 256), (1, 256, 4128, 192, 256),
                                               (1, 16384, 4128, 96, 128), (320, 4096, 1024, 4, 12), (64, 2048, 4096, 4, 16),
                                               (16, 2048, 4096, 20, 24), (8, 2048, 4096, 48, 56), (16, 1024, 2048, 48, 56),
                                               (1, 4096, 4096, 96, 128), (1, 512, 1024, 96, 192)])
def test_measured_crossings(G, N, K, lower, upper):
    """Streamed at the lower count of rows a group, tiled at the upper."""
    assert streams(lower * G, N, K, G) and not streams(upper * G, N, K, G)


@pytest.mark.parametrize("G,N,K,lower,upper", [(320, 2048, 4096, 64, 72), (320, 4096, 1024, 64, 96), (16, 2048, 4096, 192, 256),
                                               (24, 1024, 2048, 256, 384), (64, 512, 1024, 192, 256), (8, 2048, 4096, 384, 512)])
def test_short_tiles(G, N, K, lower, upper):
    """Short tiles at the lower count of rows a group, tall ones at the upper; tall ones where scale rows are no
    whole dwords."""
    f = nv.lib().moe_internal_product8_short
    f.argtypes, f.restype = [ctypes.c_int] * 5, ctypes.c_int
    assert f(lower * G, N, K, G, 256) and not f(upper * G, N, K, G, 256) and not f(lower * G, N, K + 32, G, 256)
    assert not streams(lower * G, N, K, G)


def test_extremes():
    assert streams(1, 1, 32, 1) and streams(1, 65536, 65536, 1024) and not streams(1 << 27, 65536, 65536, 1024)
