"""A pool of adapters beside one weight, fp64, and 8-bit activation
checkpoints -- oracle.

TEST INFRASTRUCTURE (see the package docstring). Row m of a batch uses adapter
a = index[m] of A [n, r, K], B [n, N, r], scale [n] (an index outside 0 .. n - 1:
none); per row the definitions are those of gemm.py. Inputs are bf16 bit
patterns; products are taken in fp64 on their exact values.

Checkpoints (blocks of 64): top = max |x|, code = nearest of 127 x / top
("int8") or nearest e4m3 value of 448 x / top ("e4m3"), ties to even, decided in
exact rational arithmetic where it matters (the quotient of two small integers
times a power of two); value = bf16_rne(fl32(code * s)), s = fl32(top / 127 or
448).
"""
import numpy as np

from .gemm import bf16_to_f64
from .nf4 import f32_to_bf16_bits


def _groups(index, n):
    index = np.asarray(index)
    return [(a, np.flatnonzero(index == a)) for a in range(n)]


def forward(x_bits, wdeq_bits, A_bits, B_bits, scale, index):
    """y [M, N]."""
    x, A, B = bf16_to_f64(x_bits), bf16_to_f64(A_bits), bf16_to_f64(B_bits)
    y = x @ bf16_to_f64(wdeq_bits).T
    for a, rows in _groups(index, len(A)):
        if len(rows):
            y[rows] += float(scale[a]) * ((x[rows] @ A[a].T) @ B[a].T)
    return y


def backward_dx(dy_bits, wdeq_bits, A_bits, B_bits, scale, index):
    """dX [M, K]."""
    dy, A, B = bf16_to_f64(dy_bits), bf16_to_f64(A_bits), bf16_to_f64(B_bits)
    dx = dy @ bf16_to_f64(wdeq_bits)
    for a, rows in _groups(index, len(A)):
        if len(rows):
            dx[rows] += float(scale[a]) * ((dy[rows] @ B[a]) @ A[a])
    return dx


def grads(x, dy_bits, A_bits, B_bits, scale, index):
    """(dA [n, r, K], dB [n, N, r]); x as fp64 values (bf16, or restored)."""
    dy, A, B = bf16_to_f64(dy_bits), bf16_to_f64(A_bits), bf16_to_f64(B_bits)
    dA, dB = np.zeros_like(A), np.zeros_like(B)
    for a, rows in _groups(index, len(A)):
        if len(rows):
            s = float(scale[a])
            dA[a] = s * ((dy[rows] @ B[a]).T @ x[rows])
            dB[a] = s * (dy[rows].T @ (x[rows] @ A[a].T))
    return dA, dB


# --------------------------------------------------------------------------
TOP = {"int8": 127, "e4m3": 448}


def e4m3_values():
    """The 256 values of the e4m3 bit patterns (OCP: bias 7, no infinity, NaN
    at 0x7F and 0xFF)."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.astype(float) - 10))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b > 127, -v, v)


def _nearest_e4m3(q):
    """e4m3 bits of each |q| <= 448, ties to the even pattern: q against the exact
    midpoints of neighbouring values (both exact in fp64)."""
    v = e4m3_values()[:127]
    mid = (v[1:] + v[:-1]) / 2
    a = np.abs(q)
    lo = np.searchsorted(mid, a, side="left")            # count of midpoints below a
    tie = (lo < len(mid)) & (mid[np.minimum(lo, len(mid) - 1)] == a)
    bits = np.where(tie & (lo % 2 == 1), lo + 1, lo)
    return (bits + 128 * np.signbit(q)).astype(np.uint8)


def pack(x_bits, fmt):
    """(codes, absmax bits) of a flat bf16 array whose size is a multiple of 64.
    top * x / max|x| is computed as (top * x) / max|x|: the product is exact in
    fp64 and the division rounds correctly, so a tie is exact and no non-tie
    becomes one."""
    bits = np.asarray(x_bits, np.uint16).reshape(-1, 64)
    x = bf16_to_f64(bits)
    bad = ~np.isfinite(x).all(axis=1)
    xs = np.where(bad[:, None], 0.0, x)
    top = np.abs(xs).max(axis=1)
    top = np.where(top < 2.0 ** -80, 0.0, top)
    live = top > 0
    q = np.where(live[:, None], TOP[fmt] * xs / np.where(live, top, 1.0)[:, None], 0.0)
    codes = np.rint(q).astype(np.int8) if fmt == "int8" else _nearest_e4m3(q)
    codes[~live] = 0
    am = f32_to_bf16_bits(top.astype(np.float32)).astype(np.uint16)
    am[bad] = 0x7FFF
    return codes.reshape(-1), am


def unpack(codes, absmax_bits, fmt):
    """bf16 bits of the restored values (NaN blocks: 0x7FFF-like NaNs)."""
    v = codes.astype(np.float32) if fmt == "int8" else e4m3_values()[codes].astype(np.float32)
    top = (np.asarray(absmax_bits, np.uint16).astype(np.uint32) << 16).view(np.float32)
    with np.errstate(invalid="ignore"):
        s = (top / np.float32(TOP[fmt])).astype(np.float32)
        return f32_to_bf16_bits((v.reshape(-1, 64) * s[:, None]).astype(np.float32).reshape(-1))
