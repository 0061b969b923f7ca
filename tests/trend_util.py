"""Helpers of the trend-network operators' GPU tests: column-major CUDA matrices with chosen
padding and offset, FP64 copies of their values, and unit roundoffs."""
import numpy as np
import torch

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
# half a unit in the last place, relative, and half the smallest subnormal
ROUND = {torch.float32: (2.0 ** -24, 2.0 ** -150), torch.float16: (2.0 ** -11, 2.0 ** -25),
         torch.bfloat16: (2.0 ** -8, 2.0 ** -134), torch.float8_e4m3fn: (2.0 ** -4, 2.0 ** -10)}


def matrix(a, dtype, pad=0, shift=0):
    """a (n x m, FP64) as a column-major CUDA matrix of dtype with leading dimension n + pad, its
    first element `shift` elements past an aligned address; padding and surroundings are NaN."""
    n, m = a.shape
    ld = n + pad
    host = torch.full((shift + m * ld + 16,), float("nan"), dtype=torch.float32)
    body = host[shift:shift + m * ld].view(m, ld)
    body[:, :n] = torch.from_numpy(np.ascontiguousarray(a.T)).float()
    flat = host.to(dtype).cuda()
    return flat[shift:shift + m * ld].view(m, ld)[:, :n].T


def vector(a):
    return torch.from_numpy(np.ascontiguousarray(a)).float().cuda()


def values(t):
    """The values of a CUDA tensor in FP64."""
    return t.detach().to(torch.float64).cpu().numpy()


def within(got, want, err, dtype):
    """|got - want| <= err (of the FP32 arithmetic) plus the rounding of `want` + err to dtype."""
    u, tiny = ROUND[dtype]
    got = values(got)
    assert got.shape == want.shape
    limit = err + u * (np.abs(want) + err) + tiny
    bad = ~(np.abs(got - want) <= limit)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(got - want) / limit, -1)), got.shape)
        raise AssertionError(f"{bad.sum()} of {bad.size} out; worst at {i}: got {got[i]}, want {want[i]}, limit {limit[i]}")
