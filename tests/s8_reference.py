"""The 8-bit linear layer's operators in 64 bits on the CPU, from their formulas, for the tests."""
from __future__ import annotations

import numpy as np
import torch

TYPES = {0: torch.float32, 1: torch.float16, 2: torch.bfloat16}
U32 = 2.0 ** -24  # a rounding to fp32: half a step


def codes(v: torch.Tensor):
    """(codes int64, scale float32) of the rows of a float64 matrix of float32 values."""
    a = v.abs().amax(1) if v.shape[1] else torch.zeros(v.shape[0], dtype=torch.float64)
    bad = ~torch.isfinite(v).all(1)
    a = torch.where(bad, 0.0, a)
    # fp32 / fp32 in numpy is the IEEE quotient
    s = torch.from_numpy(a.numpy().astype(np.float32) / np.float32(127.0))
    zero = (s == 0) | bad
    d = torch.where(zero, 1.0, s.double())
    q = torch.round(torch.where(zero[:, None], 0.0, v) / d[:, None]).clamp(-127, 127)
    s = torch.where(bad, float("nan"), s)
    return q.to(torch.int64), s


def rmsnorm(x, r, w, eps):
    """(h in the type, codes, step, scale float64)."""
    t = x.dtype
    h = x if r is None else (x.double() + r.double()).to(t)
    v = (h.double() * w.double()[None, :]).float().double()
    q, step = codes(v)
    ms = (h.double() ** 2).sum(1) / max(1, x.shape[1])
    scale = torch.where(step > 0, step.double() / torch.sqrt(ms + eps), step.double())
    return h, q, step, scale


def gemm(A, sA, B, sB, beta, C0, bias, relu, type):
    """(value float64, bound on |library - value|): A, B int8 codes; the bound counts the fp32
    roundings (the sum, two scales, beta C, two additions) and C's own."""
    acc = (A.double() @ B.double().t())
    z = acc * sA.double()[:, None] * sB.double()[None, :]
    size = z.abs()
    if beta:
        z = z + beta * C0.double()
        size = size + abs(beta) * C0.double().abs()
    if bias is not None:
        z = z + bias.double()[None, :]
        size = size + bias.double().abs()[None, :]
    if relu:
        z = torch.where(z < 0, 0.0, z)
    info = torch.finfo(TYPES[type])
    bound = 6.001 * U32 * size
    if type != 0:
        # rounding z + err to the type: half a step of it, or of its subnormals
        bound = bound + (z.abs() + bound) * (info.eps / 2) + float(info.smallest_normal) * info.eps / 2
    else:
        bound = bound + 2.0 ** -149
    return z, bound
