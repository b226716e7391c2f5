"""moe_dispatch without a workspace: taken where none is needed, refused (not an attribute error)
where one is."""
import pytest
import torch

import nvfp4_expert_layer_amd as nv
from tests.gpu_helpers import log, require_gpu


def test_binding_takes_none():
    p = nv.make_dispatch_problem(4, 16, 8, 2, 0, 8)
    assert nv.moe_dispatch_workspace_size(p) == 0
    ids, x = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="must be on the GPU"):
        nv.moe_dispatch(p, ids, x, None, None, None, None, torch.zeros(8, 16, dtype=torch.bfloat16), None)


@pytest.mark.gpu
def test_small_and_large_batches():
    require_gpu()
    log("dispatch without a workspace")
    for T in (4, 5000):
        p = nv.make_dispatch_problem(T, 16, 8, 4, 0, 8)
        ids = torch.arange(T * 4, dtype=torch.int32, device="cuda").remainder(8).view(T, 4)
        x = torch.arange(T, device="cuda").view(T, 1).remainder(251).expand(T, 16).to(torch.bfloat16).contiguous()
        rows = torch.zeros(T * 4, 16, dtype=torch.bfloat16, device="cuda")
        if nv.moe_dispatch_workspace_size(p):
            with pytest.raises(RuntimeError, match="workspace 0 < required"):
                nv.moe_dispatch(p, ids, x, None, None, None, None, rows, None)
            assert not rows.any()
        else:
            nv.moe_dispatch(p, ids, x, None, None, None, None, rows, None)
            order = ids.flatten().sort(stable=True).indices
            assert torch.equal(rows, x[order // 4])
