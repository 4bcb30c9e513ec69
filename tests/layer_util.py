"""Shared by the tests of the norm, the router and the rows' way to the experts:
device tensors between guard bytes, and 64-bit values of bf16 tensors."""
import numpy as np
import torch

GUARD = 0x5A


class Guarded:
    """A device tensor of `shape` between two runs of guard bytes."""

    def __init__(self, shape, dtype, fill=None):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        self.raw = torch.full((n + 512,), GUARD, dtype=torch.uint8, device="cuda")
        self.n = n
        self.t = self.raw[256:256 + n].view(dtype).view(shape)
        if fill is not None:
            self.t.copy_(fill)

    def intact(self):
        return bool((self.raw[:256] == GUARD).all()) and bool((self.raw[256 + self.n:] == GUARD).all())


def outs(spec):
    """{name: (shape, dtype)} -> ({name: tensor}, check that no guard was written)."""
    g = {k: Guarded(s, d) for k, (s, d) in spec.items()}
    return {k: v.t for k, v in g.items()}, lambda: [k for k, v in g.items() if not v.intact()]


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def normal(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).to(torch.bfloat16)


def generator(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def host_bits(t):
    """bf16 tensor -> uint16 patterns on the host."""
    return t.cpu().view(torch.int16).numpy().view(np.uint16)
