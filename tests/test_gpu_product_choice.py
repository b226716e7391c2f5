"""Which kernel a product takes: rows stream where a weight's bytes are the cost, and go through
tiles where streaming would walk them one pass after another on a few CUs."""
import pytest
import torch

import nvfp4_expert_layer_amd as nv
from tests.gpu_helpers import log, require_gpu
from tests.kernel_names import launched

pytestmark = pytest.mark.gpu

STREAM = {"product_resident_kernel", "product_stream_kernel"}
TILE = {"w4a16": {"a16_tile_kernel"}, "w4a4": {"mx_tile_kernel"}}


def chosen(mode, M, N, K, G=1):
    w = nv.MXFP4Weights.empty(G, N, K)
    w.codes.fill_(0x22)
    w.scales.fill_(127)
    off = torch.linspace(0, M, G + 1).int().cuda()
    out = torch.empty(M, N, device="cuda")
    a = torch.ones(M, K, dtype=torch.bfloat16, device="cuda")
    if mode == "w4a4":
        q = nv.MXFP4Rows.empty(M, K)
        nv.moe_mxfp4_quantize(a, q.codes, q.scales)
        a = q
    p = nv.make_product_problem(M, N, K, G)
    names = launched(lambda: nv.moe_mxfp4_product(p, a, w, off, out))
    assert (out == K).all()
    assert len(names) == 1, names
    return set(names)


@pytest.mark.parametrize("mode", ["w4a16", "w4a4"])
@pytest.mark.parametrize("M,N,K,G", [(512, 16, 4096, 1), (1024, 256, 4096, 1), (1200, 256, 1024, 1),
                                     (700, 512, 4096, 2), (520, 96, 7168, 1)])
def test_many_rows_of_a_narrow_product_go_through_tiles(mode, M, N, K, G):
    """Measured 1.2 to 5.2 times as long when streamed."""
    require_gpu()
    log(f"narrow product {mode} M={M} N={N} K={K} G={G}")
    assert chosen(mode, M, N, K, G) == TILE[mode]


@pytest.mark.parametrize("mode", ["w4a16", "w4a4"])
@pytest.mark.parametrize("M,N,K,G", [(1, 2048, 4096, 1), (100, 256, 4096, 1), (60, 4096, 4096, 1), (64, 512, 1024, 8),
                                     (20, 64, 8224, 1)])
def test_few_rows_stream(mode, M, N, K, G):
    require_gpu()
    log(f"few rows {mode} M={M} N={N} K={K} G={G}")
    assert chosen(mode, M, N, K, G) <= STREAM
