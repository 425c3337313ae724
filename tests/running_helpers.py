"""Plain fp64 forms of the operators that run a quantized layer, and packed test layers."""
from __future__ import annotations

import numpy as np
import torch


def pack_np(codes: np.ndarray, bits: int) -> np.ndarray:
    """LSB-first b-bit codes (m x n integers) as uint32 words, unused bits 0."""
    m, n = codes.shape
    words = (n * bits + 31) // 32
    stream = np.zeros((m, words * 32), dtype=np.uint64)
    for i in range(bits):
        stream[:, i:n * bits:bits] = (codes >> i) & 1
    place = np.uint64(1) << np.arange(32, dtype=np.uint64)
    return (stream.reshape(m, words, 32) * place).sum(2).astype(np.uint32)


def layer_np(m, n, bits, group, seed, extreme=False):
    """codes, scales, zeros (numpy) and the dequantized fp64 weights.  ``extreme``: codes and zero
    points at the ends of their range."""
    rng = np.random.default_rng(seed)
    top = (1 << bits) - 1
    size = group or n
    G = -(-n // size)
    if extreme:
        codes = rng.choice([0, top], size=(m, n))
        zeros = rng.choice([0, top], size=(m, G))
    else:
        codes = rng.integers(0, top + 1, size=(m, n))
        zeros = rng.integers(0, top + 1, size=(m, G))
    scales = np.exp(rng.standard_normal((m, G)) - 3).astype(np.float32)
    of = np.arange(n) // size
    w = scales.astype(np.float64)[:, of] * (codes - zeros[:, of])
    return codes, scales, zeros.astype(np.uint8), w


def to_cuda(codes, scales, zeros, bits):
    return (torch.from_numpy(pack_np(codes, bits).view(np.int32)).cuda(),
            torch.from_numpy(scales).cuda(), torch.from_numpy(zeros).cuda())


def check_linear(y, x64, w64, xscale=None):
    """The product against fp64, element by element and in norm.

    Every product of an input and code - zero is exact and so is the fp32 input as three parts.
    What is rounded, relative to A = sum |x| |w|: the fp32 sums (at most 3 * 256 additions inside a
    run of columns, truncated by the tensor cores to 2^-23 at worst; n / 16 scaled runs and the
    joining of at most 16 partial sums, 2^-24 each), the output (half a step), and for 8-bit rows
    the product with the row's scale (2^-24).  In norm the additions of independent terms are 16
    truncated steps a run (2^-23 each) and the scaled runs.
    """
    ref, A = x64 @ w64.T, np.abs(x64) @ np.abs(w64).T
    if xscale is not None:
        ref, A = ref * xscale[:, None], A * xscale[:, None]
    got = y.double().cpu().numpy()
    half = torch.finfo(y.dtype).eps / 2
    n = x64.shape[1]
    sums = 3 * 256 * 2.0 ** -23 + (n / 16 + 18) * 2.0 ** -24
    tiny = float(np.finfo(np.float32).tiny)
    bad = np.abs(got - ref) > half * np.abs(ref) + (1 + half) * sums * A + tiny
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], float(np.abs(got - ref).max()))
    norm = np.linalg.norm(ref)
    if norm > 0 and ref.size >= 64:
        rel = np.linalg.norm(got - ref) / norm
        assert rel <= half + 3 * 16 * 2.0 ** -23 + (n / 16 + 18) * 2.0 ** -24, rel


def norm_np(x, residual, gamma, eps, dtype):
    """(h, v, q, scale) of fp64 arrays; h rounded to ``dtype``.  A row whose largest |u| is not a
    finite positive number has codes 0."""
    h = x if residual is None else x + residual
    h = torch.from_numpy(h).to(dtype).double().numpy()
    with np.errstate(all="ignore"):
        u = h * gamma
        rstd = 1 / np.sqrt((h * h).mean(1) + eps)
        v = u * rstd[:, None]
        top = np.abs(u).max(1)
        ok = np.isfinite(top) & (top > 0)
        q = np.where(ok[:, None], np.rint(127 * u / np.where(ok, top, 1)[:, None]), 0)
        return h, v, np.nan_to_num(q).astype(np.int64), top * rstd / 127
