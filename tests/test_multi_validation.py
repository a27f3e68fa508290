"""Refusals of the multi-adapter and checkpoint calls, on the CPU: the Python
wrappers from metadata alone, the C entry points by status before any launch."""
import ctypes
import types

import pytest
import torch

from qlora_dequant_gemm_amd import _lib, ops

N, K, M, r, n = 96, 128, 4, 8, 3
bf = lambda *s: torch.empty(s, dtype=torch.bfloat16)
V = ctypes.c_void_p
FAKE, ODD = V(0x10000), V(0x10008)


def fake_weight(N, K):
    return types.SimpleNamespace(shape=(N, K), packed=torch.empty(0, dtype=torch.uint8))


def fake_pool(**kw):
    return types.SimpleNamespace(**{**dict(N=N, K=K, n=n, r=r, A=bf(n, r, K), B=bf(n, N, r),
                                           scale=torch.empty(n)), **kw})


@pytest.mark.parametrize("A,B,s,msg", [
    (bf(r, K), bf(n, N, r), torch.empty(n), "A must be a three"),
    (bf(n, r, K), bf(N, r), torch.empty(n), "B must be a three"),
    (bf(n, r, K), bf(n, N, r + 1), torch.empty(n), "B must be"),
    (bf(n, r, K), bf(n + 1, N, r), torch.empty(n), "B must be"),
    (bf(n, r, K), bf(n, N, r), torch.empty(n + 1), "scale must be"),
    (bf(n, 129, K), bf(n, N, 129), torch.empty(n), "rank 1 to 128"),
    (bf(0, r, K), bf(0, N, r), torch.empty(0), "1 to 4096 adapters"),
    (bf(n, r, K).float(), bf(n, N, r), torch.empty(n), "A must be torch.bfloat16"),
    (bf(n, r, K), bf(n, N, r), torch.empty(n), "device tensor"),
])
def test_pool_refuses(A, B, s, msg):
    with pytest.raises(ValueError, match=msg):
        ops.AdapterPool(A, B, s)


@pytest.mark.parametrize("kw,msg", [
    (dict(x=bf(M, K + 64)), "x must be"), (dict(x=bf(K)), "two-dimensional"),
    (dict(index=torch.empty(M + 1, dtype=torch.int32)), "index must be"),
    (dict(index=None), "index must be a tensor"),
    (dict(index=torch.empty(M, dtype=torch.int64)), "index must be torch.int32"),
    (dict(out=bf(M, N + 8)), "out must be"), (dict(pool=fake_pool(K=K + 64)), "adapters are for"),
    (dict(index=torch.empty(M, dtype=torch.int32)), "device tensor"),
])
def test_forward_refuses(kw, msg):
    a = {**dict(x=bf(M, K), pool=fake_pool(), index=torch.empty(M, dtype=torch.int32), out=None), **kw}
    with pytest.raises(ValueError, match=msg):
        ops.lora_fwd_multi(a["x"], fake_weight(N, K), a["pool"], a["index"], out=a["out"])


@pytest.mark.parametrize("kw,msg", [
    (dict(dy=bf(M, N + 8)), "dy must be"), (dict(out=bf(M, K + 64)), "out must be"),
    (dict(pool=fake_pool(N=N + 8)), "adapters are for"),
    (dict(index=torch.empty(1, M, dtype=torch.int32)), "index must be"),
])
def test_backward_refuses(kw, msg):
    a = {**dict(dy=bf(M, N), pool=fake_pool(), index=torch.empty(M, dtype=torch.int32), out=None), **kw}
    with pytest.raises(ValueError, match=msg):
        ops.bwd_dx_multi(a["dy"], fake_weight(N, K), a["pool"], a["index"], out=a["out"])


def test_gradients_refuse():
    ix = torch.empty(M, dtype=torch.int32)
    with pytest.raises(ValueError, match="dy must be"):
        ops.lora_grad_multi(bf(M, K), bf(M + 1, N), fake_pool(), ix)
    with pytest.raises(ValueError, match="adapters are for"):
        ops.lora_grad_multi(bf(M, K + 64), bf(M, N), fake_pool(), ix)
    with pytest.raises(ValueError, match="dA must be"):
        ops.lora_grad_multi(bf(M, K), bf(M, N), fake_pool(), ix, dA=torch.empty(n, r, K + 1))
    with pytest.raises(ValueError, match="dB must be"):
        ops.lora_grad_multi(bf(M, K), bf(M, N), fake_pool(), ix, dB=torch.empty(n, r, N))


def test_checkpoints_refuse():
    with pytest.raises(ValueError, match="fmt must be"):
        ops.act8_pack(bf(M, K), "int4")
    with pytest.raises(ValueError, match="multiple of 64"):
        ops.act8_pack(bf(M, K + 8))
    with pytest.raises(ValueError, match="non-empty"):
        ops.act8_pack(bf(0, K))
    with pytest.raises(ValueError, match="x must be torch.bfloat16"):
        ops.act8_pack(torch.empty(M, K))
    with pytest.raises(ValueError, match="device tensor"):
        ops.act8_pack(bf(M, K))
    i8 = torch.empty(M, K, dtype=torch.int8)
    with pytest.raises(ValueError, match="absmax must be"):
        ops.Act8(i8, bf(M * K // 64 + 1))
    with pytest.raises(ValueError, match="codes must be torch.uint8"):
        ops.Act8(i8, bf(M * K // 64), "e4m3")
    with pytest.raises(ValueError, match="device tensor"):
        ops.Act8(i8, bf(M * K // 64))


L = lambda: _lib.lib()


def _fwd(x=FAKE, M=16, N=64, K=64, packed=FAKE, A=FAKE, B=FAKE, s=FAKE, n=2, ix=FAKE, r=8, y=FAKE, ws=None, wsb=None):
    if wsb is None:
        wsb, ws = ops.workspace_bytes_multi(0, M, N, K, r, n), FAKE
    return L().qlora_nf4_lora_fwd_multi(x, M, N, K, packed, FAKE, FAKE, A, B, s, n, ix, r, y, ws, wsb, V(0))


def _bwd(dy=FAKE, M=16, N=64, K=64, A=FAKE, s=FAKE, n=2, ix=FAKE, r=8, dx=FAKE, ws=FAKE, wsb=0):
    return L().qlora_nf4_bwd_dx_multi(dy, M, N, K, FAKE, FAKE, FAKE, A, FAKE, s, n, ix, r, dx, ws, wsb, V(0))


def _grad(x=FAKE, fmt=2, am=V(0), dy=FAKE, M=16, N=64, K=64, A=FAKE, s=FAKE, n=2, ix=FAKE, r=8, dA=FAKE, acc=0,
          ws=FAKE, wsb=0):
    return L().qlora_lora_grad_multi(x, fmt, am, dy, M, N, K, A, FAKE, s, n, ix, r, dA, FAKE, acc, ws, wsb, V(0))


COMMON = [(dict(M=0), 2), (dict(K=96), 2), (dict(n=0), 2), (dict(n=4097), 2), (dict(r=0), 4), (dict(r=129), 4),
          (dict(A=V(0)), 1), (dict(s=V(0)), 1), (dict(ix=V(0)), 1), (dict(A=ODD), 3), (dict(s=V(0x10002)), 3),
          (dict(ix=V(0x10001)), 3), (dict(M=1 << 31), 2), (dict(N=(1 << 21) + 8), 2), (dict(wsb=16), 5),
          (dict(ws=V(0), wsb=1 << 30), 5), (dict(ws=ODD, wsb=1 << 30), 3)]


@pytest.mark.parametrize("kw,status", COMMON + [(dict(x=V(0)), 1), (dict(y=V(0)), 1), (dict(packed=V(0)), 1),
                                                (dict(x=ODD), 3), (dict(y=ODD), 3)])
def test_forward_status(kw, status):
    assert _fwd(**kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [(dict(N=12), 2), (dict(dy=V(0)), 1), (dict(dx=ODD), 3)])
def test_backward_status(kw, status):
    assert _bwd(**kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(N=12), 2), (dict(x=V(0)), 1), (dict(dA=ODD), 3), (dict(acc=2), 2), (dict(fmt=3), 6),
    (dict(fmt=2, am=FAKE), 6), (dict(fmt=0), 1), (dict(fmt=1, am=ODD), 3)])
def test_gradient_status(kw, status):
    assert _grad(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(codes=V(0)), 1), (dict(am=V(0)), 1), (dict(fmt=2), 6), (dict(N=12), 2), (dict(r=0), 4), (dict(A=V(0)), 1),
    (dict(am=ODD), 3), (dict(wsb=0), 5), (dict(acc=-1), 2)])
def test_checkpoint_gradient_status(kw, status):
    a = {**dict(codes=FAKE, am=FAKE, fmt=0, N=64, A=FAKE, r=8, acc=0, wsb=1 << 30), **kw}
    assert L().qlora_lora_grad_act8(a["codes"], a["am"], a["fmt"], FAKE, 16, a["N"], 64, a["A"], FAKE, a["r"], 1.0, FAKE,
                                    FAKE, a["acc"], FAKE, a["wsb"], V(0)) == status


def test_checkpoint_status():
    P, U = L().qlora_act8_pack, L().qlora_act8_unpack
    assert P(V(0), 64, 0, FAKE, FAKE, V(0)) == 1 and P(FAKE, 65, 0, FAKE, FAKE, V(0)) == 2
    assert P(FAKE, 0, 0, FAKE, FAKE, V(0)) == 2 and P(FAKE, 64, 2, FAKE, FAKE, V(0)) == 6
    assert P(ODD, 64, 1, FAKE, FAKE, V(0)) == 3 and P(FAKE, 1 << 43, 1, FAKE, FAKE, V(0)) == 2
    assert U(FAKE, V(0), 64, 0, FAKE, V(0)) == 1 and U(FAKE, FAKE, 64, 5, FAKE, V(0)) == 6
    assert U(FAKE, FAKE, 96, 0, FAKE, V(0)) == 2 and U(FAKE, FAKE, 64, 0, ODD, V(0)) == 3


def test_workspace_query():
    q = ops.workspace_bytes_multi
    assert q(0, 16, 64, 64, 8, 2) >= 16384 and q(4, 16, 64, 64, 8, 2) == 0 and q(0, 16, 64, 64, 8, 0) == 0
    assert q(1, 16, 12, 64, 8, 2) == 0 and q(0, 16, 12, 64, 8, 2) > 0
    # the gradients' lists and partial sums grow with the batch, not with M times n
    assert q(2, 4096, 4096, 4096, 16, 4096) < 8 * q(2, 4096, 4096, 4096, 16, 1)
    for op in range(4):
        assert q(op, 333, 136, 320, 24, 5) % 256 == 0


def test_gradients_of_long_batches_split_nothing():
    """A split product of a chunk needs one of 4096 arrival counters, so a batch
    of more than 2048 chunks has none: its workspace holds the rows' lists, t and
    u, and the items' sums, and no partial sums of t and u (130 KB a chunk)."""
    M, K, N, r = 132000, 576, 64, 8
    chunks = M // 64 + 2
    items = 2 * (M // 64) * 4 * 256 * 16 * 4 // 17
    need = _lib.lib().qlora_workspace_bytes_multi(2, M, N, K, r, 2)
    assert 0 < need < 16384 + chunks * 64 * (4 + 2 * 3 * 16 * 2) + items + (1 << 20)
    assert 0 < _lib.lib().qlora_workspace_bytes_multi(3, M, N, K, r, 1) < need + (1 << 20)


def test_limits_of_rows_and_values():
    size = _lib.lib().qlora_workspace_bytes_multi
    for op in range(4):
        assert size(op, (1 << 28) - 1, 8, 64, 1, 1) > 0 and size(op, 1 << 28, 8, 64, 1, 1) == 0
    P, U = _lib.lib().qlora_act8_pack, _lib.lib().qlora_act8_unpack
    assert P(FAKE, 1 << 37, 0, FAKE, FAKE, V(0)) == 2 and U(FAKE, FAKE, 1 << 37, 0, FAKE, V(0)) == 2
