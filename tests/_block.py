"""Shared helpers of the tests of the operators around the layer: guarded outputs, error bounds
and plain 64-bit forms."""
import torch

import weight_sequence_layers_b200 as ttt

F64 = torch.float64
U32 = 2.0 ** -24  # half a step of float32, relative
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
GUARD = 64        # elements of the pattern on each side of a guarded output


def half(dtype):
    """Half a rounding step of a type, relative to the value."""
    return torch.finfo(dtype).eps / 2


class Out:
    """An output tensor between two guard regions; every element starts as NaN."""

    def __init__(self, *shape, dtype=torch.float32):
        n = 1
        for s in shape:
            n *= s
        pad = GUARD * 4 // torch.empty((), dtype=dtype).element_size()  # keeps 16-byte alignment
        self.buf = torch.full((n + 2 * pad,), float("nan"), dtype=dtype, device="cuda")
        self.buf[:pad], self.buf[pad + n:] = 7.0, 7.0
        self.t = self.buf[pad:pad + n].view(shape)
        self.pad, self.n = pad, n

    def check(self):
        assert bool((self.buf[:self.pad] == 7.0).all()) and \
            bool((self.buf[self.pad + self.n:] == 7.0).all()), "written outside the output"
        return self.t


def assert_within(name, got, ref, bound):
    """|got - ref| <= bound + half a step of got's type, elementwise; ref and bound in float64."""
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    if not got.numel():
        return
    g = got.to(F64)
    assert bool(torch.isfinite(g).all()), f"{name}: not finite"
    # a rounding is relative to the value rounded, which is within bound of ref; the smallest
    # normal of bf16 and float32 covers results that underflow
    tol = bound + half(got.dtype) * (ref.abs() + bound) + 2.0 ** -126
    over = (g - ref).abs() - tol
    worst = float(over.max())
    assert worst <= 0, (name, worst, float((g - ref).abs().max()), int((over > 0).sum()), got.numel())


def rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=torch.float32, std=1.0, mean=0.0):
    return torch.empty(shape, device="cuda").normal_(mean, std, generator=g).to(dtype)


def sync_ok():
    torch.cuda.synchronize()
    assert ttt.ttt_get_device_error() == ttt.OK


def workspace(n):
    """A workspace full of NaN bytes, so that a kernel relying on its contents shows."""
    return torch.full((max(n, 16),), 255, dtype=torch.uint8, device="cuda")
