"""moe_route and its gradient where a wave takes several tokens and a block several waves."""
import numpy as np
import pytest
import torch

from tests.gpu_helpers import log, require_gpu
from tests.test_gpu_topk import check, check_gradient, draw, run

pytestmark = pytest.mark.gpu


def sampled(T):
    """The first and last tokens, and every 97th."""
    return sorted({*range(9), *range(0, T, 97), *range(T - 9, T)})


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [1027, 5001, 16389])
@pytest.mark.parametrize("k", [8, 16, 17, 20])
@pytest.mark.parametrize("renormalize", [True, False])
def test_several_tokens_a_wave(kind, T, k, renormalize):
    """One, two and four tokens a wave, segments of 16 and 32 lanes, the last batch short; tokens without
    experts among the others."""
    require_gpu()
    log(f"route batches {kind} T={T} k={k} renormalize={renormalize}")
    logits, bias = draw(T, 160, torch.float32, T + k)
    logits[[1, 6, T - 2]] = -float("inf")                        # no expert at all
    logits[[2, T - 5], 5:] = float("nan")                        # five
    for kw in (dict(), dict(groups=8, top_groups=4)):
        for b in (None, bias):
            ids, w = check(logits, b, k, kind, sampled(T), renormalize=renormalize, scale=2.5, **kw)
            assert (ids[[1, 6, T - 2]] == -1).all() and (w[[1, 6, T - 2]] == 0).all()
            # a choice among 160 experts is whole everywhere else
            rest = np.setdiff1d(np.arange(T), [1, 6, T - 2, 2, T - 5])
            assert (ids[rest] >= 0).all() and (w[rest] > 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,k", [(1500, 320, 8), (1025, 7, 3), (1090, 1000, 32)])
def test_gradient_of_several_waves(dtype, kind, renormalize, T, E, k):
    """Four waves a block, each with a row of its own in LDS; the last block's some without one."""
    require_gpu()
    log(f"route gradient waves {dtype} {kind} renormalize={renormalize} T={T} E={E} k={k}")
    logits, bias = draw(T, E, dtype, T + E)
    ids = torch.from_numpy(run(logits, bias, k, kind)[0])
    ids[::50] = -1
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(k))
    got = check_gradient(logits, ids, dw, kind, renormalize, 2.5)
    assert (got[::50] == 0).all()
