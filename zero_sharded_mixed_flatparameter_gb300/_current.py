"""The current device and stream as numbers.

torch's own helpers below its public functions cost a tenth of a microsecond
where those build an object for each call; a torch without them has the public
ones used.
"""

from __future__ import annotations

import torch


def _public_stream(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or _public_stream
