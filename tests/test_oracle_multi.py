"""Pins of the multi-adapter and checkpoint oracle against things other than
itself: the single-adapter oracle, differences of the forward, torch's e4m3
type, rational brute force around every tie."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import gemm, multi
from oracle.nf4 import f32_to_bf16_bits


def bits(a):
    return f32_to_bf16_bits(np.asarray(a, np.float32)).astype(np.uint16)


def case(M, N, K, r, n, seed):
    g = np.random.Generator(np.random.PCG64(seed))
    return (bits(g.standard_normal((M, K))), bits(g.standard_normal((M, N))), bits(g.standard_normal((N, K)) * 0.1),
            bits(g.standard_normal((n, r, K)) * 0.3), bits(g.standard_normal((n, N, r)) * 0.3),
            (g.random(n) + 0.5).astype(np.float32), g.integers(-1, n + 1, M).astype(np.int32))


def test_rows_agree_with_the_single_adapter_oracle():
    x, dy, w, A, B, s, idx = case(23, 12, 64, 4, 3, 0)
    y, dx = multi.forward(x, w, A, B, s, idx), multi.backward_dx(dy, w, A, B, s, idx)
    for m, a in enumerate(idx):
        one = (A[a], B[a], float(s[a]) * 4, 4) if 0 <= a < 3 else ()
        assert np.allclose(y[m], gemm.lora_forward(x[m:m + 1], w, *one)[0], rtol=1e-12)
        assert np.allclose(dx[m], gemm.backward_dx(dy[m:m + 1], w, *one)[0], rtol=1e-12)
    dA, dB = multi.grads(gemm.bf16_to_f64(x), dy, A, B, s, idx)
    for a in range(3):
        rows = idx == a
        oA, oB = gemm.lora_grads(x[rows], dy[rows], A[a], B[a], float(s[a]) * 4, 4)
        assert np.allclose(dA[a], oA, rtol=1e-10) and np.allclose(dB[a], oB, rtol=1e-10)


def test_gradients_are_differences_of_the_forward():
    x, dy, w, A, B, s, idx = case(17, 8, 64, 3, 2, 1)
    f = gemm.bf16_to_f64
    dA, dB = multi.grads(f(x), dy, A, B, s, idx)
    g = np.random.Generator(np.random.PCG64(2))

    def loss(Av, Bv):                         # <dY, y>, fp64 adapters
        y = f(x) @ f(w).T
        for m, a in enumerate(idx):
            if 0 <= a < 2:
                y[m] += float(s[a]) * ((f(x)[m] @ Av[a].T) @ Bv[a].T)
        return float((f(dy) * y).sum())
    EA, EB = g.standard_normal(A.shape), g.standard_normal(B.shape)
    h = 0.5                                    # the loss is quadratic: a central difference is exact
    d = (loss(f(A) + h * EA, f(B) + h * EB) - loss(f(A) - h * EA, f(B) - h * EB)) / (2 * h)
    assert np.isclose(d, (dA * EA).sum() + (dB * EB).sum(), rtol=1e-9)
    # dX against differences in x
    dx = multi.backward_dx(dy, w, A, B, s, idx)
    base = f(x)
    for _ in range(5):
        m, k = int(g.integers(17)), int(g.integers(64))
        def y_of(v):
            xx = base[m].copy()
            xx[k] = v
            out = xx @ f(w).T
            a = idx[m]
            if 0 <= a < 2:
                out = out + float(s[a]) * ((xx @ f(A)[a].T) @ f(B)[a].T)
            return float(out @ f(dy)[m])
        assert np.isclose(y_of(base[m, k] + 1) - y_of(base[m, k]), dx[m, k], rtol=1e-8, atol=1e-8)


def test_an_adapter_without_rows_gets_zero():
    x, dy, w, A, B, s, _ = case(5, 8, 64, 3, 4, 3)
    dA, dB = multi.grads(gemm.bf16_to_f64(x), dy, A, B, s, np.array([0, 2, 2, -1, 9]))
    assert not dA[1].any() and not dB[3].any() and dA[2].any()


def test_e4m3_table_is_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, multi.e4m3_values(), equal_nan=True)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_codes_are_the_nearest_in_rational_arithmetic(fmt):
    g = np.random.Generator(np.random.PCG64(4))
    x = g.standard_normal(64 * 24).astype(np.float32)
    x.reshape(24, 64)[3, 5] = 80.0
    b = bits(x).reshape(24, 64)
    # ties: the block's largest is 127 (448) quarter steps, others on half steps
    top = bits([multi.TOP[fmt] / 4.0])[0]
    b[7, 0], b[7, 1:33] = top, bits((np.arange(32) + 0.5) / 4)
    b[8, 0], b[8, 1:33] = top | 0x8000, bits(-(np.arange(32) + 0.5) / 64)
    # half the largest is a tie for int8 whatever the block
    for i in range(9, 20):
        m = np.argmax(b[i] & 0x7FFF)
        b[i, (m + 1) % 64] = (b[i, m] & 0x7FFF) - 0x80
    codes, am = multi.pack(b.reshape(-1), fmt)
    val = multi.e4m3_values()
    for i in range(24):
        top = Fraction(float(gemm.bf16_to_f64(b[i] & 0x7FFF).max()))
        assert (am[i].astype(np.uint32) << 16).view(np.float32) == float(top)
        for j in range(64):
            q = Fraction(float(gemm.bf16_to_f64(b[i, j:j + 1])[0])) * multi.TOP[fmt] / top
            c = codes[64 * i + j]
            if fmt == "int8":
                assert c == round(q)                       # Python rounds ties to even
            else:
                d = [abs(abs(q) - Fraction(float(v))) for v in val[:127]]
                best = [k for k in range(127) if d[k] == min(d)]
                k = best[0] if len(best) == 1 else [k for k in best if k % 2 == 0][0]
                assert (c & 127) == k


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_restored_values_are_close_and_ends_exact(fmt):
    g = np.random.Generator(np.random.PCG64(5))
    b = bits(g.standard_normal(64 * 200) * np.exp(g.standard_normal(64 * 200)))
    codes, am = multi.pack(b, fmt)
    x = gemm.bf16_to_f64(b).reshape(-1, 64)
    y = gemm.bf16_to_f64(multi.unpack(codes, am, fmt)).reshape(-1, 64)
    top = np.abs(x).max(1, keepdims=True)
    assert np.array_equal(np.abs(y).max(1, keepdims=True), top)
    step = top / 254 if fmt == "int8" else np.maximum(np.abs(x) / 16, top / 448 / 1024)
    assert (np.abs(x - y) <= step * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(x)).all()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_special_blocks(fmt):
    b = np.zeros((5, 64), np.uint16)
    b[1, 3], b[1, 4] = 0x7F80, 0x3F80                      # an infinity
    b[2, 60] = 0xFFC1                                      # a NaN
    b[3] = bits(np.full(64, 2.0 ** -81))                   # below 2^-80
    b[4, 7] = bits([2.0 ** -80])[0]
    codes, am = multi.pack(b.reshape(-1), fmt)
    y = gemm.bf16_to_f64(multi.unpack(codes, am, fmt)).reshape(5, 64)
    assert not y[0].any() and np.isnan(y[1]).all() and np.isnan(y[2]).all() and not y[3].any()
    assert y[4, 7] == 2.0 ** -80
