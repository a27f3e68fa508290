"""GPU tests of the pool of adapters (forward, backward to the input, adapter
gradients) and of 8-bit activation checkpoints, against the fp64 oracle.

Bounds, per element, from the arithmetic of the kernels:
  * a product of c terms accumulated in fp32 is off by at most c 2^-23 sum |terms|
    (2^-24 per addition, twice that for an accumulator that truncates);
  * t = bf16(x . A^T) and u = bf16(dY . B) of the forward and the backward are off by
    2^-8 relative, so s |t| |B| 2^-8 reaches the output;
  * the bf16 output adds 2^-8 relative;
  * the gradients carry t and u as three bf16 numbers (2^-24 relative, the
    fp32 rounding itself) and are fp32.
Codes, constants and restored values of checkpoints are bit-exact.
"""
import numpy as np
import pytest
import torch

import synth
from oracle import gemm, multi, nf4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from qlora_dequant_gemm_amd import ops
    return ops


def dev(a):
    t = torch.from_numpy(np.ascontiguousarray(a))
    if a.dtype == np.uint16:
        t = t.view(torch.int16).view(torch.bfloat16)
    return t.cuda()


def bits(a):
    return nf4.f32_to_bf16_bits(np.asarray(a, np.float32))


def host(t):
    """fp64 values of a device tensor."""
    return t.detach().to(torch.float64).cpu().numpy()


def host_bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


f64 = gemm.bf16_to_f64


def rows_of(kind, M, n, seed):
    """int32 [M] adapters: "one" adapter; "runs" of requests (some on the base
    alone, some indexes out of range); "mixed" row by row; "none"; "last" row only."""
    g = np.random.Generator(np.random.PCG64(seed))
    if kind == "one":
        return np.full(M, n - 1, np.int32)
    if kind == "none":
        return np.full(M, -1, np.int32)
    if kind == "last":
        return np.concatenate([np.full(M - 1, n + 3), [0]]).astype(np.int32)
    if kind == "mixed":
        return g.integers(-1, n + 1, M).astype(np.int32)
    ids = g.integers(-1, n + 1, 9)
    ids[4] = -2 ** 31
    cuts = np.sort(g.integers(0, M + 1, 8))
    return np.repeat(ids, np.diff(np.concatenate([[0], cuts, [M]]))).astype(np.int32)


class Case:
    def __init__(self, ops, M, N, K, r, n, kind, seed):
        g = np.random.Generator(np.random.PCG64(seed))
        self.M, self.N, self.K, self.r, self.n = M, N, K, r, n
        self.w = synth.weight(N, K, seed)
        self.qw = ops.quantize_weight(dev(self.w))
        packed, q, step, _ = nf4.quantize_all(self.w)
        self.wd = nf4.dequantize(packed, q, step).reshape(N, K)
        self.x = bits(g.standard_normal((M, K)))
        self.dy = bits(g.standard_normal((M, N)) * 0.1)
        self.A = bits(g.standard_normal((n, r, K)) * K ** -0.5)
        self.B = bits(g.standard_normal((n, N, r)) * 0.1)
        self.s = (g.random(n) * 1.5 + 0.5).astype(np.float32)
        self.idx = rows_of(kind, M, n, seed + 1)
        self.pool = ops.AdapterPool(dev(self.A), dev(self.B), dev(self.s))
        self.index = dev(self.idx)

    def per_row(self, P):
        """|P| of the row's adapter (zeros for none), fp64 [M, ...]."""
        ok = (self.idx >= 0) & (self.idx < self.n)
        a = np.abs(f64(P))
        out = a[np.where(ok, self.idx, 0)]
        out[~ok] = 0
        return out, np.where(ok, self.s[np.where(ok, self.idx, 0)], 0)[:, None]

    def check_fwd(self, y):
        ref = multi.forward(self.x, self.wd, self.A, self.B, self.s, self.idx)
        aA, s = self.per_row(self.A)
        aB, _ = self.per_row(self.B)
        ax = np.abs(f64(self.x))
        T = np.einsum("mk,mrk->mr", ax, aA)
        base = ax @ np.abs(f64(self.wd)).T
        lora = s * np.einsum("mr,mnr->mn", T, aB)
        A, B = f64(self.A), f64(self.B)
        ok = np.where((self.idx >= 0) & (self.idx < self.n), self.idx, 0)
        t = np.abs(np.einsum("mk,mrk->mr", f64(self.x), A[ok]))
        e = (self.K + self.r + 4) * 2.0 ** -23 * (base + lora) + 2.0 ** -8 * s * np.einsum("mr,mnr->mn", t, aB)
        self.bounded(y, ref, e, 2.0 ** -8)

    def check_bwd(self, dx):
        ref = multi.backward_dx(self.dy, self.wd, self.A, self.B, self.s, self.idx)
        aA, s = self.per_row(self.A)
        aB, _ = self.per_row(self.B)
        ad = np.abs(f64(self.dy))
        U = np.einsum("mn,mnr->mr", ad, aB)
        ok = np.where((self.idx >= 0) & (self.idx < self.n), self.idx, 0)
        u = np.abs(np.einsum("mn,mnr->mr", f64(self.dy), f64(self.B)[ok]))
        mag = ad @ np.abs(f64(self.wd)) + s * np.einsum("mr,mrk->mk", U, aA)
        e = (self.N + self.r + 4) * 2.0 ** -23 * mag + 2.0 ** -8 * s * np.einsum("mr,mrk->mk", u, aA)
        self.bounded(dx, ref, e, 2.0 ** -8)

    def check_grads(self, dA, dB, x=None, dA0=0.0, dB0=0.0):
        x = f64(self.x) if x is None else x
        rA, rB = multi.grads(x, self.dy, self.A, self.B, self.s, self.idx)
        ax = np.abs(x)
        ad = np.abs(f64(self.dy))
        A, B = np.abs(f64(self.A)), np.abs(f64(self.B))
        dA, dB = host(dA), host(dB)
        for a in range(self.n):
            rows = self.idx == a
            s, c = float(self.s[a]), int(rows.sum())
            U = ad[rows] @ B[a]
            T = ax[rows] @ A[a].T
            eA = (self.N + 2 * c + 16) * 2.0 ** -23 * s * (U.T @ ax[rows])
            eB = (self.K + 2 * c + 16) * 2.0 ** -23 * s * (ad[rows].T @ T)
            self.bounded(dA[a], rA[a] + dA0, eA + 2.0 ** -23 * abs(dA0), 2.0 ** -24)
            self.bounded(dB[a], rB[a] + dB0, eB + 2.0 ** -23 * abs(dB0), 2.0 ** -24)

    @staticmethod
    def bounded(got, ref, e, rounding):
        got = got if isinstance(got, np.ndarray) else host(got)
        assert got.shape == ref.shape
        over = np.abs(got - ref) - (e + rounding * (np.abs(ref) + e))
        at = np.unravel_index(np.argmax(np.where(np.isnan(over), np.inf, over)), over.shape)
        assert over[at] <= 0, f"at {at}: got {got[at]}, expected {ref[at]} within {e[at]}"


SHAPES = [
    # M, N, K, r, n, rows
    (1, 64, 64, 8, 1, "one"),
    (1, 40, 128, 16, 3, "one"),
    (2, 72, 192, 5, 2, "mixed"),
    (15, 264, 320, 16, 20, "mixed"),
    (16, 128, 256, 4, 3, "none"),
    (17, 320, 512, 16, 4, "last"),
    (33, 8, 64, 32, 5, "mixed"),
    (64, 520, 1024, 16, 64, "mixed"),
    (65, 256, 576, 24, 3, "runs"),
    (130, 264, 320, 128, 2, "runs"),
    (255, 96, 256, 64, 7, "runs"),
    (300, 512, 768, 16, 4, "runs"),
    (300, 264, 128, 100, 5, "mixed"),
    (515, 264, 320, 32, 9, "runs"),
    (777, 136, 1216, 1, 300, "mixed"),
]


@pytest.mark.parametrize("M,N,K,r,n,kind", SHAPES + [(4, 2056, 4160, 128, 5, "mixed"),
                                                          (4, 4096, 1024, 16, 4, "mixed"), (40, 37, 128, 8, 3, "runs"), (260, 301, 320, 12, 3, "mixed"),
                                                     (5, 1, 2112, 16, 2, "mixed"), (48, 200, 4160, 16, 30, "mixed"),
                                                     # a contraction split over workgroups: the tiled kernel, ragged and whole
                                                     (1100, 264, 2112, 16, 6, "runs"), (1030, 520, 2048, 40, 40, "mixed"),
                                                     # its other rank groups; up to four rows
                                                     (1100, 264, 320, 100, 3, "runs"), (1090, 40, 192, 24, 5, "mixed"),
                                                     (1200, 520, 64, 80, 4, "runs"), (1, 4104, 1088, 100, 2, "one"),
                                                     (2, 520, 4096, 64, 2, "mixed"), (4, 264, 2112, 33, 9, "mixed"),
                                                     (3, 72, 64, 16, 3, "last"), (4, 136, 320, 16, 2, "none")])
def test_forward(qops, M, N, K, r, n, kind):
    c = Case(qops, M, N, K, r, n, kind, 100 + M)
    c.check_fwd(qops.lora_fwd_multi(dev(c.x), c.qw, c.pool, c.index))


@pytest.mark.parametrize("M,N,K,r,n,kind", SHAPES + [(130, 1544, 320, 24, 5, "runs"), (70, 2056, 192, 64, 33, "mixed"),
                                                     (600, 4104, 576, 16, 3, "runs"), (3, 8200, 64, 8, 2, "mixed")])
def test_backward(qops, M, N, K, r, n, kind):
    c = Case(qops, M, N, K, r, n, kind, 200 + M)
    c.check_bwd(qops.bwd_dx_multi(dev(c.dy), c.qw, c.pool, c.index))


@pytest.mark.parametrize("M,N,K,r,n,kind", SHAPES + [(60, 2056, 4160, 80, 3, "runs"), (1300, 1032, 2112, 16, 20, "mixed"),
                                                     # past the batch that lists itself; many adapters, most without rows
                                                     (8200, 40, 64, 8, 5, "mixed"), (9001, 24, 128, 33, 3, "runs"),
                                                     (100, 40, 64, 4, 4096, "mixed"), (8192, 8, 64, 4, 2, "runs")])
def test_gradients(qops, M, N, K, r, n, kind):
    c = Case(qops, M, N, K, r, n, kind, 300 + M)
    ws = qops.Workspace("cuda")
    dA, dB = qops.lora_grad_multi(dev(c.x), dev(c.dy), c.pool, c.index, ws=ws)
    c.check_grads(dA, dB)
    eA, eB = qops.lora_grad_multi(dev(c.x), dev(c.dy), c.pool, c.index, ws=ws)
    assert torch.equal(dA, eA) and torch.equal(dB, eB)
    dA.fill_(0.5)
    dB.fill_(-0.25)
    qops.lora_grad_multi(dev(c.x), dev(c.dy), c.pool, c.index, dA=dA, dB=dB, accumulate=True, ws=ws)
    c.check_grads(dA, dB, dA0=0.5, dB0=-0.25)


def test_gradients_of_long_runs(qops):
    """Adapters of many items (summed partials) beside one of a single row and
    one without rows."""
    c = Case(qops, 4500, 72, 128, 16, 4, "one", 9)
    c.idx = np.concatenate([np.full(3000, 2), np.full(1499, 0), [3]]).astype(np.int32)
    c.idx = c.idx[np.random.Generator(np.random.PCG64(1)).permutation(4500)]
    dA, dB = qops.lora_grad_multi(dev(c.x), dev(c.dy), c.pool, dev(c.idx))
    c.check_grads(dA, dB)
    assert not dA[1].any() and not dB[1].any()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("M,N,K,r,n,kind", [SHAPES[0], SHAPES[2], SHAPES[3], SHAPES[8], SHAPES[9], SHAPES[13]])
def test_gradients_from_checkpoints(qops, M, N, K, r, n, kind, fmt):
    c = Case(qops, M, N, K, r, n, kind, 400 + M)
    kept = qops.act8_pack(dev(c.x), fmt)
    codes, am = multi.pack(c.x.reshape(-1), fmt)
    x = f64(multi.unpack(codes, am, fmt)).reshape(M, K)
    dA, dB = qops.lora_grad_multi(kept, dev(c.dy), c.pool, c.index)
    c.check_grads(dA, dB, x=x)
    # the restored values give the same gradients, bit for bit
    eA, eB = qops.lora_grad_multi(qops.act8_unpack(kept), dev(c.dy), c.pool, c.index)
    assert torch.equal(dA, eA) and torch.equal(dB, eB)
    # one adapter for every row
    c.idx = np.zeros(M, np.int32)
    alpha = float(c.s[0]) * r
    c.s[0] = np.float32(alpha) / np.float32(r)
    dA, dB = qops.lora_grad(kept, dev(c.dy), dev(c.A[0]), dev(c.B[0]), alpha)
    one = Case.__new__(Case)
    one.__dict__.update(c.__dict__, n=1, A=c.A[:1], B=c.B[:1], s=c.s[:1])
    one.check_grads(dA[None], dB[None], x=x)
    dA.fill_(2.0), dB.fill_(1.0)
    qops.lora_grad(kept, dev(c.dy), dev(c.A[0]), dev(c.B[0]), alpha, dA=dA, dB=dB, accumulate=True)
    one.check_grads(dA[None], dB[None], x=x, dA0=2.0, dB0=1.0)


def test_single_adapter_checkpoint_gradients_over_many_items(qops):
    c = Case(qops, 2100, 264, 192, 16, 1, "one", 11)
    kept = qops.act8_pack(dev(c.x))
    x = host(qops.act8_unpack(kept))
    dA, dB = qops.lora_grad(kept, dev(c.dy), dev(c.A[0]), dev(c.B[0]), float(c.s[0]) * 16)
    c.check_grads(dA[None], dB[None], x=x)


# ---------------------------------------------------------------------------
def ckpt_blocks():
    """Blocks with the places where a code can go wrong: every bf16 bit pattern
    as a value, ties of both formats, extremes, and special blocks."""
    g = np.random.Generator(np.random.PCG64(6))
    out = [np.arange(65536, dtype=np.uint16).reshape(-1, 64)]            # neighbours share a block
    x = bits(g.standard_normal((400, 64)))
    x[::7] = bits(g.standard_normal((58, 64)) * 3e38 / 5)                # the largest magnitudes
    x[1::7] = bits(g.standard_normal((57, 64)) * 2.0 ** -79)             # either side of 2^-80
    x[2::7, 9] = x[2::7, 30] | 0x7000                                    # one large value
    for i in range(3, 400, 7):                                           # half the largest: a tie
        m = np.argmax(x[i] & 0x7FFF)
        x[i, (m + 1) % 64] = (x[i, m] & 0x7FFF) - 0x80
    for i, top in enumerate((127.0, 448.0, 254.0, 112.0)):               # half steps of the codes
        x[4 + 7 * i, 0] = bits([top / 4])[0]
        x[4 + 7 * i, 1:] = bits(np.arange(63) / 8 - 2)
    x[5, 3], x[12, 60], x[19] = 0x7F80, 0xFFC1, 0
    x[26] = 0x8000
    return np.concatenate(out + [x])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_checkpoint_is_bit_exact(qops, fmt):
    b = ckpt_blocks()
    for rows in (1, 3, 17, len(b)):
        x = b[-rows:]
        kept = qops.act8_pack(dev(x), fmt)
        codes, am = multi.pack(x.reshape(-1), fmt)
        got = kept.codes.cpu().numpy().reshape(-1)
        assert np.array_equal(got, codes.reshape(-1)), np.flatnonzero(got != codes.reshape(-1))[:8]
        assert np.array_equal(host_bits(kept.absmax), am)
        y, ref = host_bits(qops.act8_unpack(kept)).reshape(-1), multi.unpack(codes, am, fmt)
        nan = np.isnan(f64(ref))
        assert np.array_equal(np.isnan(f64(y)), nan) and np.array_equal(y[~nan], ref[~nan])
    assert kept.nbytes * 64 == x.size * 66


def test_checkpoint_shapes_and_buffers(qops):
    x = torch.randn(3, 5, 192, device="cuda").to(torch.bfloat16)
    kept = qops.act8_pack(x, "e4m3")
    assert kept.shape == (3, 5, 192) and kept.absmax.numel() == 45
    guard = torch.full((3 * 5 * 192 + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = guard[:-64].view(3, 5, 192)
    assert qops.act8_unpack(kept, out=out) is out
    assert torch.equal(out, qops.act8_unpack(qops.Act8(kept.codes, kept.absmax, "e4m3")))
    assert (guard[-64:] == 7.0).all()


# ---------------------------------------------------------------------------
@pytest.mark.parametrize("M", [4, 8, 300, 1100])
def test_bad_numbers_stay_with_their_rows(qops, M):
    """NaN and infinities in one adapter, its scale or a row of x reach only the
    rows and gradients that use them."""
    c = Case(qops, M, 264, 320, 16, 4, "mixed", 21)
    c.idx[:4] = [0, 1, 2, 3]
    clean = qops.lora_fwd_multi(dev(c.x), c.qw, c.pool, dev(c.idx))
    cdx = qops.bwd_dx_multi(dev(c.dy), c.qw, c.pool, dev(c.idx))
    cA, cB = qops.lora_grad_multi(dev(c.x), dev(c.dy), c.pool, dev(c.idx))
    A, B, s, x, dy = c.A.copy(), c.B.copy(), c.s.copy(), c.x.copy(), c.dy.copy()
    A[1, 3, 17] = 0x7FC0
    B[1, 200, 5] = 0x7F80
    s[2] = np.inf
    x[3, 11] = 0x7F80
    dy[3, 7] = 0xFF80
    pool = qops.AdapterPool(dev(A), dev(B), dev(s))
    y = qops.lora_fwd_multi(dev(x), c.qw, pool, dev(c.idx))
    dx = qops.bwd_dx_multi(dev(dy), c.qw, pool, dev(c.idx))
    dA, dB = qops.lora_grad_multi(dev(x), dev(dy), pool, dev(c.idx))
    fine = torch.from_numpy((c.idx != 1) & (c.idx != 2) & (np.arange(M) != 3)).cuda()
    assert torch.equal(y[fine], clean[fine]) and torch.equal(dx[fine], cdx[fine])
    assert torch.equal(dA[0], cA[0]) and torch.equal(dB[0], cB[0])
    assert not torch.isfinite(y[3]).all() and not torch.isfinite(dA[3]).all() and not torch.isfinite(dB[1]).all()
    kept = qops.act8_pack(dev(x))
    dA, dB = qops.lora_grad_multi(kept, dev(dy), pool, dev(c.idx))
    assert not torch.isfinite(dA[3]).all() and torch.isfinite(dA[0]).all()


@pytest.mark.parametrize("M,N,K", [(4, 264, 320), (40, 264, 320), (300, 72, 320), (300, 264, 2112), (700, 1032, 576), (1100, 264, 320)])
def test_bad_rows_stay_apart(qops, M, N, K):
    """Rows of NaN in x or dY change no bit of their neighbours, whose products end
    inside a step of the contraction, nor of other adapters' gradients."""
    c = Case(qops, M, N, K, 16, 4, "mixed", 23)
    bad = np.arange(M) % 5 == 2
    c.idx[bad], c.idx[~bad] = 3, c.idx[~bad] % 3
    index, fine = dev(c.idx), torch.from_numpy(~bad).cuda()
    res = []
    for v in (0, 0x7FC0):
        c.x[bad], c.dy[bad] = v, v
        x, dy = dev(c.x), dev(c.dy)
        dA, dB = qops.lora_grad_multi(x, dy, c.pool, index)
        res.append((qops.lora_fwd_multi(x, c.qw, c.pool, index)[fine], qops.bwd_dx_multi(dy, c.qw, c.pool, index)[fine],
                    dA[:3], dB[:3]))
    for a, b in zip(*res):
        assert torch.equal(a, b)


def test_outputs_end_where_they_end(qops):
    """Nothing is written past the outputs; a workspace full of NaN changes nothing."""
    c = Case(qops, 83, 136, 320, 24, 3, "runs", 31)
    ws = qops.Workspace("cuda")
    for op in range(3):
        ws.get(qops.workspace_bytes_multi(op, 83, 136, 320, 24, 3))
    ws.buf[16384:].fill_(0xFF)
    g = torch.full((83 * 320 + 512,), 3.0, dtype=torch.bfloat16, device="cuda")
    y = g[:83 * 136].view(83, 136)
    qops.lora_fwd_multi(dev(c.x), c.qw, c.pool, c.index, out=y, ws=ws)
    c.check_fwd(y)
    assert (g[83 * 136:] == 3.0).all()
    dx = g[:83 * 320].view(83, 320)
    ws.buf[16384:].fill_(0xFF)
    qops.bwd_dx_multi(dev(c.dy), c.qw, c.pool, c.index, out=dx, ws=ws)
    c.check_bwd(dx)
    assert (g[83 * 320:] == 3.0).all()
    f = torch.full((3 * 24 * (320 + 136) + 256,), 3.0, device="cuda")
    dA, dB = f[:3 * 24 * 320].view(3, 24, 320), f[3 * 24 * 320:-256].view(3, 136, 24)
    ws.buf[16384:].fill_(0xFF)
    qops.lora_grad_multi(dev(c.x), dev(c.dy), c.pool, c.index, dA=dA, dB=dB, ws=ws)
    c.check_grads(dA, dB)
    assert (f[-256:] == 3.0).all()
    assert not ws.buf[:16384].any()


def step(ops, c, x, dy, pool, index, ws, bufs):
    """One training step of a linear in a batch of several adapters, with its
    input kept in 8 bits: forward, backward, gradients."""
    y = ops.lora_fwd_multi(x, c.qw, pool, index, out=bufs[0], ws=ws)
    kept = ops.act8_pack(x)
    dx = ops.bwd_dx_multi(dy, c.qw, pool, index, out=bufs[1], ws=ws)
    dA, dB = ops.lora_grad_multi(kept, dy, pool, index, dA=bufs[2], dB=bufs[3], ws=ws)
    return y, kept, dx, dA, dB


@pytest.mark.parametrize("M,kind", [(3, "mixed"), (48, "mixed"), (333, "runs"), (1100, "runs")])
def test_a_step_eager_streams_and_replayed(qops, M, kind):
    c = Case(qops, M, 264, 320, 16, 5, kind, 41)
    x, dy = dev(c.x), dev(c.dy)
    bf, f32 = torch.bfloat16, torch.float32
    new = lambda: [torch.empty(s, dtype=t, device="cuda") for s, t in
                   [((M, 264), bf), ((M, 320), bf), ((5, 16, 320), f32), ((5, 264, 16), f32)]]
    ws = qops.Workspace("cuda")
    y, kept, dx, dA, dB = step(qops, c, x, dy, c.pool, c.index, ws, new())
    c.check_fwd(y)
    c.check_bwd(dx)
    c.check_grads(dA, dB, x=host(qops.act8_unpack(kept)))
    eager = [t.clone() for t in (y, dx, dA, dB)]
    # on another stream, with a workspace of its own, beside calls on this one
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ws2 = qops.Workspace("cuda")
        got2 = step(qops, c, x, dy, c.pool, c.index, ws2, new())
    got1 = step(qops, c, x, dy, c.pool, c.index, ws, new())
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for got in (got1, got2):
        assert all(torch.equal(a, b) for a, b in zip((got[0], got[2], got[3], got[4]), eager))
    # captured once, replayed with other inputs and eager calls between
    bufs = new()
    xs, ds, ix = x.clone(), dy.clone(), c.index.clone()
    gws = qops.Workspace("cuda")
    with torch.cuda.stream(side):
        step(qops, c, xs, ds, c.pool, ix, gws, bufs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(qops, c, xs, ds, c.pool, ix, gws, bufs)
    for k in range(4):
        other = rows_of(("runs", "mixed", "none", "one")[k], M, 5, 50 + k)
        xs.copy_(x.roll(k, 0)), ds.copy_(dy.roll(k, 0)), ix.copy_(dev(other))
        for b in bufs:
            b.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want = step(qops, c, xs, ds, c.pool, ix, ws, new())
        assert all(torch.equal(a, b) for a, b in zip(bufs, (want[0], want[2], want[3], want[4])))


def test_gradient_matches_differences_of_the_forward(qops):
    """<dY, y(A + hE) - y(A - hE)> / 2h against <dA, E> (y is linear in A), with
    every number a multiple of a power of two so that the forward is exact."""
    M, N, K, r, n = 32, 64, 64, 8, 2
    g = np.random.Generator(np.random.PCG64(51))
    c = Case(qops, M, N, K, r, n, "mixed", 51)
    x, dy = bits(g.integers(-1, 2, (M, K))), bits(g.integers(-1, 2, (M, N)))
    A, B = g.integers(-1, 2, (n, r, K)), bits(g.integers(-1, 2, (n, N, r)) / 4)
    E = g.integers(-1, 2, (n, r, K))
    s = np.ones(n, np.float32)
    c.qw.qscale.zero_()                                   # the base is zero
    at = lambda Av: host(qops.lora_fwd_multi(dev(x), c.qw, qops.AdapterPool(dev(bits(Av)), dev(B), dev(s)), c.index))
    d = ((at(A + E) - at(A - E)) * f64(dy)).sum() / 2
    dA, _ = qops.lora_grad_multi(dev(x), dev(dy), qops.AdapterPool(dev(bits(A)), dev(B), dev(s)), c.index)
    # t is an integer below 2^8 (|x . A| <= 128) and y a multiple of 1/4 below 2^8 with at most
    # 8 significant bits or rounded by 2^-8 relative: the sum of |dY| |y| 2^-8 bounds the difference
    slack = 2.0 ** -8 * (np.abs(at(A + E)) + np.abs(at(A - E))).sum() / 2
    assert abs(d - (host(dA) * E).sum()) <= slack
    dB = qops.lora_grad_multi(dev(x), dev(dy), qops.AdapterPool(dev(bits(A)), dev(B), dev(s)), c.index)[1]
    rA, rB = multi.grads(f64(x), dy, bits(A), B, s, c.idx)
    assert np.array_equal(host(dA), rA) and np.array_equal(host(dB), rB)     # all exact in fp32


@pytest.mark.parametrize("M,N,K,r", [(4, 11008, 4096, 16), (700, 4096, 11008, 16), (1500, 11008, 4096, 64)])
def test_full_size(qops, M, N, K, r):
    """Every output at layer sizes: relative Frobenius error of bf16 outputs at
    most 5e-3 (2^-8 output rounding and 2^-8 of the adapter term), of fp32
    gradients at most 1e-5, against fp64 products of the same bf16 values."""
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    n = 6
    bf = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(torch.bfloat16)
    qw = qops.quantize_weight(bf(N, K, std=0.02))
    x, dy, A, B = bf(M, K), bf(M, N, std=0.01), bf(n, r, K, std=K ** -0.5), bf(n, N, r, std=0.05)
    s = torch.rand(n, generator=g, device="cuda") + 0.5
    index = (torch.arange(M, device="cuda") * 8 // M - 1).to(torch.int32)
    pool = qops.AdapterPool(A, B, s)
    W = qops.dequant(qw).double()
    y, dx = x.double() @ W.t(), dy.double() @ W
    rA, rB = torch.zeros(n, r, K, dtype=torch.float64, device="cuda"), torch.zeros(n, N, r, dtype=torch.float64, device="cuda")
    for a in range(n):
        rows = torch.nonzero(index == a)[:, 0]
        xa, da, sa = x[rows].double(), dy[rows].double(), s[a].double()
        y[rows] += sa * (xa @ A[a].double().t()) @ B[a].double().t()
        dx[rows] += sa * (da @ B[a].double()) @ A[a].double()
        rA[a], rB[a] = sa * (da @ B[a].double()).t() @ xa, sa * da.t() @ (xa @ A[a].double().t())
    fro = lambda got, ref: float((got.double() - ref).norm() / ref.norm())
    assert fro(qops.lora_fwd_multi(x, qw, pool, index), y) < 5e-3
    assert fro(qops.bwd_dx_multi(dy, qw, pool, index), dx) < 5e-3
    dA, dB = qops.lora_grad_multi(x, dy, pool, index)
    assert fro(dA, rA) < 1e-5 and fro(dB, rB) < 1e-5


def test_gradients_of_many_chunks(qops):
    """More chunks (2064) than half the arrival counters, K at least three times
    N: the last rows' adapter, the pool's and the single one's gradients, and a
    second call on the workspace that the first one left."""
    M, N, K, r, n = 132000, 64, 576, 8, 3
    g = np.random.Generator(np.random.PCG64(71))
    x = (torch.from_numpy(g.standard_normal((M, K)).astype(np.float32))).to(torch.bfloat16)
    dy = torch.from_numpy(g.standard_normal((M, N)).astype(np.float32) * 0.1).to(torch.bfloat16)
    A, B = bits(g.standard_normal((n, r, K)) * K ** -0.5), bits(g.standard_normal((n, N, r)) * 0.1)
    s = np.array([1.0, 0.5, 2.0], np.float32)
    idx = np.repeat(np.array([1, -1, 2], np.int32), [100000, 1000, M - 101000])
    pool, ws = qops.AdapterPool(dev(A), dev(B), dev(s)), qops.Workspace("cuda")
    for fmt in (None, "int8"):
        xd = x.cuda() if fmt is None else qops.act8_pack(x.cuda(), fmt)
        xv = x if fmt is None else qops.act8_unpack(xd).cpu()
        x64, d64 = xv.double().numpy(), dy.double().numpy()
        first = qops.lora_grad_multi(xd, dy.cuda(), pool, dev(idx), ws=ws)
        again = qops.lora_grad_multi(xd, dy.cuda(), pool, dev(idx), ws=ws)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
        single = []
        if fmt:
            single = [(*qops.lora_grad(xd, dy.cuda(), dev(A[2]), dev(B[2]), alpha=8.0, ws=ws), slice(0, M), 2, 1.0)]
        got = [(first[0][a], first[1][a], idx == a, a, float(s[a])) for a in range(n)] + single
        for dA, dB, rows, a, sc in got:
            xr, dr, Aa, Ba = x64[rows], d64[rows], f64(A[a]), f64(B[a])
            U, T = dr @ Ba, xr @ Aa.T
            aU, aT = np.abs(dr) @ np.abs(Ba), np.abs(xr) @ np.abs(Aa).T
            c = len(xr)
            Case.bounded(dA, sc * U.T @ xr, (N + 2 * c + 16) * 2.0 ** -23 * sc * (aU.T @ np.abs(xr)), 2.0 ** -24)
            Case.bounded(dB, sc * dr.T @ T, (K + 2 * c + 16) * 2.0 ** -23 * sc * (np.abs(dr).T @ aT), 2.0 ** -24)


@pytest.mark.parametrize("M", [1, 4, 20, 300])
def test_an_infinity_stays_one(qops, M):
    """An infinite t or u gives infinities of the formula's sign, not NaN."""
    c = Case(qops, M, 264, 320, 16, 2, "one", 31)
    c.A[1, 3, 0] = 0x7F80                                     # +inf
    c.x[:, 0] = 0x3F80                                        # t[3] = +inf
    pool = qops.AdapterPool(dev(c.A), dev(c.B), dev(c.s))
    y = host(qops.lora_fwd_multi(dev(c.x), c.qw, pool, c.index))
    sign = np.sign(f64(c.B[1, :, 3]))
    assert (y[:, sign != 0] == np.inf * sign[sign != 0]).all()
    dA, dB = qops.lora_grad_multi(dev(c.x[:1]), dev(c.dy[:1]), pool, c.index[:1])
    sign = np.sign(f64(c.dy[0]))
    assert (host(dB[1])[sign != 0, 3] == np.inf * sign[sign != 0]).all()
    assert torch.isfinite(dB[1][:, :3]).all() and torch.isfinite(dA).all()


# Offsets past 2^31 elements and 2^32 bytes. Each is compared with the same rows
# or adapters alone, whose own results the tests above pin: t and u may round
# differently where another number of ranges adds them (2^-8 of the LoRA term,
# which is below a fifth of the largest output here), outputs once more (2^-8).
def near(got, ref, rel):
    got, ref = got.float(), ref.float()
    assert (got - ref).abs().max() <= rel * ref.abs().max(), float((got - ref).abs().max() / ref.abs().max())


def test_offsets_of_a_large_pool(qops):
    n, r, K, N = 2100, 128, 8192, 64
    g = torch.Generator("cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.float32)
    qw, qt = qops.quantize_weight(rnd(N, K) * 0.02), qops.quantize_weight(rnd(K, N) * 0.02)
    ends = [0, n - 1]
    wide, small = torch.zeros(n, r, K, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, N, r, dtype=torch.bfloat16, device="cuda")
    wide[ends] = (rnd(2, r, K) * K ** -0.5).bfloat16()
    small[ends] = (rnd(2, N, r) * 0.1).bfloat16()
    scale = torch.ones(n, device="cuda")
    pool = qops.AdapterPool(wide, small, scale)               # A past 2^31 elements
    few = qops.AdapterPool(wide[ends].contiguous(), small[ends].contiguous(), scale[:2].contiguous())
    turn = qops.AdapterPool(small.view(n, r, N), wide.view(n, K, r), scale)          # B past them
    fewt = qops.AdapterPool(small[ends].view(2, r, N).contiguous(), wide[ends].view(2, K, r).contiguous(), scale[:2].contiguous())
    for M in (3, 20, 300, 1100):
        idx = torch.arange(M, device="cuda", dtype=torch.int32) % 2
        big = idx * (n - 1)
        x, dy = rnd(M, K).bfloat16(), rnd(M, N).bfloat16()
        near(qops.lora_fwd_multi(x, qw, pool, big), qops.lora_fwd_multi(x, qw, few, idx), 2.0 ** -7)
        near(qops.bwd_dx_multi(dy, qw, pool, big), qops.bwd_dx_multi(dy, qw, few, idx), 2.0 ** -7)
        near(qops.lora_fwd_multi(dy, qt, turn, big), qops.lora_fwd_multi(dy, qt, fewt, idx), 2.0 ** -7)
        near(qops.bwd_dx_multi(x, qt, turn, big), qops.bwd_dx_multi(x, qt, fewt, idx), 2.0 ** -7)
        dA, dB = qops.lora_grad_multi(x, dy, pool, big)       # dA 8.8 GB
        fA, fB = qops.lora_grad_multi(x, dy, few, idx)
        near(dA[ends], fA, 2.0 ** -18)
        near(dB[ends], fB, 2.0 ** -18)
        assert not dA[1:-1].any() and not dB[1:-1].any()
        del dA, dB


def test_offsets_of_a_large_batch(qops):
    M, K, N, r, n, tail = 270000, 8192, 64, 16, 3, 300
    g = torch.Generator("cuda").manual_seed(6)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.float32)
    qw, qt = qops.quantize_weight(rnd(N, K) * 0.02), qops.quantize_weight(rnd(K, N) * 0.02)
    x = torch.randn((M, K), generator=g, device="cuda", dtype=torch.bfloat16)        # 4.4 GB
    dy = torch.randn((M, N), generator=g, device="cuda", dtype=torch.bfloat16)
    A, B = (rnd(n, r, K) * K ** -0.5).bfloat16(), (rnd(n, N, r) * 0.1).bfloat16()
    scale = torch.ones(n, device="cuda")
    pool = qops.AdapterPool(A, B, scale)
    turn = qops.AdapterPool(B.view(n, r, N), A.view(n, K, r), scale)
    idx = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    idx[-tail:] = (torch.arange(tail, device="cuda") // 64 % n).int()
    xt, dt, it = x[-tail:], dy[-tail:], idx[-tail:].contiguous()
    near(qops.lora_fwd_multi(x, qw, pool, idx)[-tail:], qops.lora_fwd_multi(xt, qw, pool, it), 2.0 ** -7)
    near(qops.bwd_dx_multi(x, qt, turn, idx)[-tail:], qops.bwd_dx_multi(xt, qt, turn, it), 2.0 ** -7)
    near(qops.lora_fwd_multi(dy, qt, turn, idx)[-tail:], qops.lora_fwd_multi(dt, qt, turn, it), 2.0 ** -7)   # y 4.4 GB
    near(qops.bwd_dx_multi(dy, qw, pool, idx)[-tail:], qops.bwd_dx_multi(dt, qw, pool, it), 2.0 ** -7)
    for a, b in zip(qops.lora_grad_multi(x, dy, pool, idx), qops.lora_grad_multi(xt, dt, pool, it)):
        near(a, b, 2.0 ** -18)
    kept, small = qops.act8_pack(x, "e4m3"), qops.act8_pack(xt, "e4m3")
    assert torch.equal(kept.codes[-tail:], small.codes)
    assert torch.equal(kept.absmax[-tail * K // 64:].view(torch.int16), small.absmax.view(torch.int16))
    assert torch.equal(qops.act8_unpack(kept)[-tail:], qops.act8_unpack(small))
    for a, b in zip(qops.lora_grad_multi(kept, dy, pool, idx), qops.lora_grad_multi(small, dt, pool, it)):
        near(a, b, 2.0 ** -18)
