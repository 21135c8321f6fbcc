"""Helpers of the GPU tests of the operators around the expert layer."""
from __future__ import annotations

import numpy as np
import torch

from _moe_helpers import host

PAD = 256            # bytes behind an output that must stay as they were


class Out:
    """An output tensor with PAD bytes of a pattern behind it; every byte holds it before the call."""

    def __init__(self, shape, dtype):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        self.raw = torch.full((n + PAD,), 0xA5, dtype=torch.uint8, device="cuda")
        self.n = n
        self.t = self.raw[:n].view(dtype).view(shape)

    def bits(self) -> np.ndarray:
        """The values' bits (or the values, for int32 and float32), after checking what is behind them."""
        assert bool((self.raw[self.n:] == 0xA5).all()), "written behind the output"
        t = self.t
        if t.dtype in (torch.bfloat16, torch.uint16, torch.int16):
            return host(t.view(torch.int16)).view(np.uint16)
        if t.dtype == torch.float8_e4m3fn:
            return host(t.view(torch.uint8))
        return host(t)


def up(a: np.ndarray) -> torch.Tensor:
    """numpy -> GPU; uint16 is taken as bf16 bits."""
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        return torch.from_numpy(a.view(np.int16)).cuda().view(torch.bfloat16)
    return torch.from_numpy(a).cuda()


def same_f32(a, b) -> bool:
    return np.array_equal(np.asarray(a, np.float32).view(np.uint32), np.asarray(b, np.float32).view(np.uint32))
