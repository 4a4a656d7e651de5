"""Shared by the GPU tests of the feature operators: types, device copies and
the comparison against error bounds that the tests derive element by element.

u(t) = eps(t) / 2 bounds one rounding to type t relative to the value;
U = 2^-24 is the same for the fp32 arithmetic inside the kernels."""

import numpy as np
import torch

from gpu_util import dev, say

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# half the spacing of the subnormals (bf16 and fp32: far below any bound here)
TINY = {"bf16": 0.0, "fp16": 2.0 ** -25, "fp32": 0.0}


def u(t):
    return torch.finfo(TYPES[t]).eps / 2


def rounded(a, t):
    """A numpy array rounded to type t: the CPU tensor and its fp64 values."""
    x = torch.from_numpy(np.ascontiguousarray(a)).to(TYPES[t])
    return x, x.double().numpy()


def put(x):
    return x.to(dev())


def strided(x, pad, shift=0):
    """The same values on the GPU with rows pad elements longer, starting `shift` elements in."""
    rows, cols = x.shape
    big = torch.full((rows, cols + pad), float("nan"), dtype=x.dtype, device=dev())
    view = big[:, shift:shift + cols]
    view.copy_(x)
    return view


def host(x):
    torch.cuda.synchronize()
    return x.double().cpu().numpy()


def within(got, want, bound, what):
    got = host(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, f"{what}: {got.shape} vs {want.shape}"
    nan = np.isnan(want)
    assert (np.isnan(got) == nan).all(), f"{what}: NaN in other places"
    err = np.where(nan, 0.0, np.abs(np.where(nan, 0, got) - np.where(nan, 0, want)))
    bound = np.broadcast_to(bound, want.shape)
    ratio = err / np.maximum(np.where(nan, 1.0, bound), 1e-300)
    say(f"    {what}: max err {err.max():.3e}, {ratio.max():.3f} of its bound")
    assert (ratio <= 1).all(), f"{what}: {int((ratio > 1).sum())} values past their bound, worst {ratio.max():.3f} at " \
        f"{np.unravel_index(ratio.argmax(), ratio.shape)}"
