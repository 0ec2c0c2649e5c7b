"""Plain block-scaled FP8 (one scale per 128 values) on the CPU: quantisation step by step in numpy
fp32, products in fp64.  Test infrastructure only."""
import numpy as np
import torch

MAX = {0: 448.0, 1: 57344.0}
F8 = {0: torch.float8_e4m3fn, 1: torch.float8_e5m2}


def blocks(n):
    return (n + 127) // 128


def scale_of(amax, fmt):
    """(scale, stored factor) in fp32 from an fp32 array of block maxima."""
    amax = np.asarray(amax, np.float32)
    safe = np.where(amax > 0, np.maximum(amax, np.float32(2.0 ** -100)), np.float32(1))
    sc = np.where(amax > 0, np.float32(MAX[fmt]) / safe, np.float32(1)).astype(np.float32)
    return sc, (np.float32(1) / sc).astype(np.float32)


def magnitude(x):
    return np.where(np.isfinite(x), np.abs(x), np.float32(0))


def encode(x, scale, fmt):
    """Codes of fl32(x * scale): nearest, ties to even, saturating; NaN stays NaN."""
    with np.errstate(over="ignore", invalid="ignore"):
        y = torch.from_numpy((x * scale).astype(np.float32))
    return y.clamp(-MAX[fmt], MAX[fmt]).to(F8[fmt]).view(torch.uint8).numpy()


def rows(x, fmt):
    """codes [R, C], factors [C/128, R] of fp32 x."""
    R, C = x.shape
    q, s = np.zeros((R, C), np.uint8), np.zeros((blocks(C), R), np.float32)
    for b in range(blocks(C)):
        part = x[:, 128 * b:128 * b + 128]
        sc, s[b] = scale_of(magnitude(part).max(1), fmt)
        q[:, 128 * b:128 * b + 128] = encode(part, sc[:, None], fmt)
    return q, s


def cols(x, fmt, offsets=None):
    """Transposed codes [C, T] and factors [T/128, C]; groups padded to multiples of 128.  Also how many of the T
    columns belong to a group's blocks."""
    R, C = x.shape
    off = [0, R] if offsets is None else list(offsets)
    G = len(off) - 1
    T = (R + 127 * min(G, R)) // 128 * 128
    q, s = np.zeros((C, T), np.uint8), np.zeros((T // 128, C), np.float32)
    b = 0
    for lo, hi in zip(off[:-1], off[1:]):
        for r in range(lo, hi, 128):
            part = x[r:min(r + 128, hi)].T
            sc, s[b] = scale_of(magnitude(part).max(1), fmt)
            q[:, 128 * b:128 * b + part.shape[1]] = encode(part, sc[:, None], fmt)
            b += 1
    return q, s, 128 * b


def weight(w, fmt):
    """codes [R, C], factors [C/128, R/128]."""
    R, C = w.shape
    q, s = np.zeros((R, C), np.uint8), np.zeros((blocks(C), blocks(R)), np.float32)
    for i in range(blocks(R)):
        for j in range(blocks(C)):
            at = (slice(128 * i, 128 * i + 128), slice(128 * j, 128 * j + 128))
            sc, s[j, i] = scale_of(magnitude(w[at]).max(), fmt)
            q[at] = encode(w[at], sc, fmt)
    return q, s


def values(q, fmt, s, per):
    """fp64 numbers of codes q [R, K] with factors s [K/128, R/per]."""
    v = torch.from_numpy(np.ascontiguousarray(q)).view(F8[fmt]).to(torch.float64).numpy()
    f = np.repeat(np.asarray(s, np.float64).T, per, 0)[:v.shape[0]]
    return v * np.repeat(f, 128, 1)[:, :v.shape[1]]


def bound(ref, absum, K, dtype):
    """What |D - ref| may be.  Per block: 128 exact products summed in fp32 on the tensor cores (2^-20 of the sum of
    magnitudes, the tensor-core bound of the other GEMM tests), the product of the two factors rounded (2^-24), one
    fused multiply-add into the running sum (2^-24 of the magnitudes so far, blocks(K) of them, and 8 joins of a split
    sum and a bias add at most), then one rounding to the output type (half a step)."""
    half = torch.finfo(dtype).eps / 2
    e = (2.0 ** -20 + (blocks(K) + 10) * 2.0 ** -24) * absum
    return half * np.abs(ref) + (1 + half) * e + 1e-38


def check(D, ref, absum, K, what):
    got = D.detach().double().cpu().numpy()
    b = bound(ref, absum, K, D.dtype)
    bad = ~(np.abs(got - ref) <= b)
    if bad.any():
        at = tuple(np.argwhere(bad)[0])
        raise AssertionError("%s: %d of %d out of bound, first %s: got %r, reference %r, bound %r" % (
            what, bad.sum(), bad.size, at, got[at], ref[at], b[at]))
