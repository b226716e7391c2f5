"""Which of the library's kernels a call launches (test infrastructure): names from a trace of
the device."""
import re

import torch
from torch.profiler import ProfilerActivity, profile


def launched(call):
    """Names, without template arguments, of the library's kernels that `call` launches, in order
    of their start."""
    torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CUDA], acc_events=True) as p:
        call()
        torch.cuda.synchronize()
    found = []
    for e in p.events():
        m = re.search(r"\bmoe::(\w+)\b", e.name)
        if m:
            found.append((e.time_range.start, m.group(1)))
    return [n for _, n in sorted(found)]
