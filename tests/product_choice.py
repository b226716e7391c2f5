"""Which kernels a product takes (test infrastructure): the rule that the library's launches use."""
import ctypes

import torch

import nvfp4_expert_layer_amd as nv


def streams(mode, M, N, K, G=1, stride=None, cus=None):
    """Whether the product ("w4a16", "w4a4") or its gradient ("backward") of M rows takes the
    streaming kernels; False: the tiles.  stride: of the row operand, by default its width; cus: by
    default the device's."""
    f = nv.lib().moe_internal_product_streams
    f.argtypes = [ctypes.c_int] * 4 + [ctypes.c_int64] + [ctypes.c_int] * 3
    f.restype = ctypes.c_int
    if stride is None:
        stride = N if mode == "backward" else K
    if cus is None:
        cus = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    return bool(f(M, N, K, G, stride, mode == "w4a4", mode == "backward", cus))
