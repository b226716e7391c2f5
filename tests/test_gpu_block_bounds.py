"""What include/moe_block.h states of the operators' ranges: the norm's magnitudes, SwiGLU's far gates, MXFP8's
smallest values; and that a call writes its outputs alone."""
import numpy as np
import pytest
import torch

import nvfp4_expert_layer_amd as nv
from tests.gpu_helpers import log, require_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24                                                   # half a step of fp32, relative


def norm(x, eps):
    T, d = x.shape
    y, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
    nv.moe_norm(nv.make_norm_problem(T, d, eps, x.dtype, torch.float32), x, None, torch.ones(d, device="cuda"), None, y,
                None, rstd)
    return y.double().cpu().numpy(), rstd.double().cpu().numpy()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [1, 7, 64, 100, 4096, 10000, 65536])
def test_norm_magnitudes(dtype, d):
    """Rows of alike magnitudes up to 2^64 / sqrt(d), beyond which rstd and y are 0; with eps 0 down to 2^-63, and
    rstd Inf where every square vanishes."""
    require_gpu()
    log(f"norm magnitudes {dtype} d={d}")
    top = 2.0 ** 64 / d ** 0.5
    m = torch.tensor([0.98 * top, 1.01 * top, 2.0 ** -62, 2.0 ** -80]).to(dtype)      # (bf16 rounds by 2^-9)
    sign = torch.where(torch.arange(d) % 3 == 0, -1.0, 1.0).to(dtype)
    x = m.unsqueeze(1) * sign
    y, rstd = norm(x.cuda(), 0.0)
    want = 1 / np.abs(m.double().numpy())
    # up to 64 squares in a row a thread, 6 steps of a wave, 16 waves: 86 roundings, halved by the root; four more
    for i in (0, 2):
        assert abs(rstd[i] - want[i]) <= 50 * U * want[i]
        assert (np.abs(y[i] - sign.double().numpy()) <= 60 * U + torch.finfo(dtype).eps / 2).all()
    assert rstd[1] == 0 and (y[1] == 0).all() and rstd[3] == np.inf
    # beside eps a mean square below 2^-25 of it leaves no trace
    _, rstd = norm(torch.full((1, d), 2.0 ** -24, dtype=dtype, device="cuda"), 2.0 ** -20)
    assert rstd[0] == 2.0 ** 10
