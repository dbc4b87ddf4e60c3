"""Inputs of the microscaled 4-bit tests: seeded matrices as the oracle stores them."""
import numpy as np
import torch

import bit_weight_only_quantize_amd as w4
import oracle

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def bf16(a):
    """fp64 array -> the bf16 tensor (host) of its nearest values."""
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(torch.bfloat16)


def matrix(shape, seed, std=0.02, spread=0.5):
    """(codes, scale, fp64 values) of a quantized matrix [N][K], or of a stack of them."""
    rng = np.random.default_rng(seed)
    x = std * rng.normal(size=shape) * np.exp(spread * rng.normal(size=shape[:-1] + (1,)))
    c, s = oracle.mx4_quantize(x.astype(np.float32))
    return c, s, oracle.mx4_values(c, s)


def integers(shape, seed, lo=126, hi=129):
    """The same with random codes and scales of a few binades: values are multiples of 2^(lo - 128)."""
    rng = np.random.default_rng(seed)
    c = rng.integers(0, 256, size=shape[:-1] + (shape[-1] // 2,)).astype(np.uint8)
    s = rng.integers(lo, hi, size=shape[:-1] + (shape[-1] // 32,)).astype(np.uint8)
    return c, s, oracle.mx4_values(c, s)


def device(codes, scale):
    """The library's matrix (or stack) of these arrays."""
    E = codes.shape[0] if codes.ndim == 3 else 1
    return w4.QuantizedMatrix("mx4_g32", codes.shape[-2], 2 * codes.shape[-1], torch.from_numpy(codes).cuda(),
                              torch.from_numpy(scale).cuda(), None, E)


def strided(t, slack):
    """A device copy of the host rows t with `slack` more columns (of NaN) between them."""
    if not slack:
        return t.cuda()
    wide = torch.full((t.shape[0], t.shape[1] + slack), float("nan"), dtype=t.dtype)
    wide[:, :t.shape[1]] = t
    return wide.cuda()[:, :t.shape[1]]


def product(x, w):
    """x w^T in fp64 by the GPU's library, and the same of the magnitudes."""
    a, b = (torch.as_tensor(v, dtype=torch.float64).cuda() for v in (x, w))
    return (a @ b.t()).cpu(), (a.abs() @ b.abs().t()).cpu()
