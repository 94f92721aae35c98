"""Pins of the dense-operator oracle (layer norm, linear layer, dropout) and host checks of the
library's entry points; no GPU."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import dense as od
from token_sparse_long_b200 import _lib


@pytest.fixture(scope="module")
def lib():
    from token_sparse_long_b200 import build
    build.build()
    return _lib.load()


def _rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def test_philox_known_answers():
    # known-answer vectors published with the generator (philox4x32, 10 rounds)
    f = 0xFFFFFFFF
    for ctr, key, want in (
            ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            ((f, f, f, f), (f, f), (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
             (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))):
        got = od.philox4x32_10(np.array([ctr], np.uint64), key)[0]
        assert tuple(int(v) for v in got) == want


def test_dropout_mask_rate_and_keys():
    m = od.dropout_mask(np.arange(4096), 512, 0.25, 7, 9)
    # 2^21 Bernoulli(3/4) draws: five standard deviations of the mean
    assert abs(m.mean() - 0.75) < 5 * np.sqrt(0.25 * 0.75 / m.size)
    assert abs(np.corrcoef(m[:, 0], m[:, 1])[0, 1]) < 5 / np.sqrt(4096)
    for other in (od.dropout_mask(np.arange(4096), 512, 0.25, 8, 9), od.dropout_mask(np.arange(4096), 512, 0.25, 7, 10),
                  od.dropout_mask(np.arange(4096), 512, 0.25, 7, 9 + (1 << 32)),
                  od.dropout_mask(np.arange(4096), 512, 0.25, 7 + (1 << 32), 9)):
        assert 0.3 < (other != m).mean() < 0.45  # 2 * 0.25 * 0.75 = 0.375
    assert (od.dropout_mask(np.arange(100, 200), 512, 0.25, 7, 9) == m[100:200]).all()
    assert (od.dropout_mask([3], 77, 0.25, 7, 9) == m[3:4, :77]).all()
    assert od.dropout_mask(np.arange(4), 64, 0.0, 1, 1).all() and not od.dropout_mask(np.arange(4), 64, 1.0, 1, 1).any()


def _diff(f, x, dy, eps=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += eps
        b[i] -= eps
        g[i] = ((f(a) - f(b)) * dy).sum() / (2 * eps)
    return g


def test_layernorm_against_torch_and_differences():
    r = _rng(0)
    x, dy, ga, be = r.normal(size=(4, 9)) + 2.0, r.normal(size=(4, 9)), r.normal(size=9), r.normal(size=9)
    y, mean, rstd = od.layernorm_fwd(x, ga, be)
    t = [torch.tensor(v, requires_grad=True) for v in (x, ga, be)]
    ty = torch.nn.functional.layer_norm(t[0], (9,), t[1], t[2], eps=1e-5)
    ty.backward(torch.tensor(dy))
    np.testing.assert_allclose(y, ty.detach().numpy(), rtol=1e-12, atol=1e-12)
    dx, dg, db = od.layernorm_bwd(dy, x, mean, rstd, ga)
    for got, want in zip((dx, dg, db), t):
        np.testing.assert_allclose(got, want.grad.numpy(), rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(dx, _diff(lambda v: od.layernorm_fwd(v, ga, be)[0], x, dy), rtol=1e-6, atol=1e-8)
    np.testing.assert_allclose(dg, _diff(lambda v: od.layernorm_fwd(x, v, be)[0], ga, dy), rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("kind", ["none", "relu", "gelu", "silu"])
def test_linear_against_torch_and_differences(kind):
    r = _rng(1)
    x, w, b, res, dy = (r.normal(size=s) for s in ((5, 6), (7, 6), (7,), (5, 7), (5, 7)))
    y, z = od.linear_fwd(x, w, b, kind, res)
    t = [torch.tensor(v, requires_grad=True) for v in (x, w, b)]
    f = {"none": lambda v: v, "relu": torch.relu, "gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu}[kind]
    ty = f(t[0] @ t[1].T + t[2]) + torch.tensor(res)
    ty.backward(torch.tensor(dy))
    np.testing.assert_allclose(y, ty.detach().numpy(), rtol=1e-12, atol=1e-12)
    dx, dw, db, _ = od.linear_bwd(dy, x, w, kind, z)
    for got, want in zip((dx, dw, db), t):
        np.testing.assert_allclose(got, want.grad.numpy(), rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(dx, _diff(lambda v: od.linear_fwd(v, w, b, kind)[0], x, dy), rtol=1e-5, atol=1e-7)
    np.testing.assert_allclose(dw, _diff(lambda v: od.linear_fwd(x, v, b, kind)[0], w, dy), rtol=1e-5, atol=1e-7)


# ------------------------------------------------------------------ refusals before any launch
N0 = ctypes.c_void_p(0)
P = [ctypes.c_void_p(1 << 20 << i) for i in range(12)]  # far apart, 16-byte aligned
F32, BF16 = _lib.F32, _lib.BF16


def ln_fwd(lib, **k):
    a = dict(x=P[0], ldx=64, S=8, h=64, idx=N0, n=N0, blk=1, rows=8, g=P[1], b=P[2], wdt=F32, eps=1e-5, dt=F32, y=P[3],
             ldy=64, mean=P[4], rstd=P[5])
    a.update(k)
    return lib.jenga_layernorm_fwd(*a.values(), None)


def ln_bwd(lib, **k):
    a = dict(dy=P[0], ldy=64, x=P[1], ldx=64, S=8, h=64, idx=N0, n=N0, blk=1, rows=8, mean=P[2], rstd=P[3], g=P[4],
             wdt=F32, dres=N0, ldr=0, dt=F32, dx=P[5], ldd=64, dg=P[6], db=P[7], acc=0, ws=P[8], wsb=1 << 20)
    a.update(k)
    return lib.jenga_layernorm_bwd(*a.values(), None)


def lin_fwd(lib, **k):
    a = dict(x=P[0], ldx=64, w=P[1], ldw=64, bias=P[2], bdt=F32, act=0, res=N0, ldr=0, M=8, N=64, K=64, n=N0, blk=1,
             y=P[3], ldy=64, pre=N0, ldp=0, ws=P[4], wsb=1 << 20)
    a.update(k)
    return lib.jenga_linear_fwd(*a.values(), None)


def lin_bwd(lib, **k):
    a = dict(dy=P[0], ldy=64, x=P[1], ldx=64, w=P[2], ldw=64, act=1, pre=P[3], ldp=64, M=8, N=64, K=64, n=N0, blk=1,
             dx=P[4], ldd=64, dw=P[5], lddw=64, db=P[6], acc=0, ws=P[7], wsb=1 << 20)
    a.update(k)
    return lib.jenga_linear_bwd(*a.values(), None)


def drop(lib, **k):
    a = dict(x=P[0], ldx=64, res=N0, ldr=0, rows=8, cols=64, idx=N0, n=N0, blk=1, row0=0, p=0.1, seed=1, off=1, dt=F32,
             y=P[1], ldy=64)
    a.update(k)
    return lib.jenga_dropout(*a.values(), None)


@pytest.mark.parametrize("fn,bad", [
    (ln_fwd, dict(x=N0)), (ln_fwd, dict(y=N0)), (ln_fwd, dict(ldx=63)), (ln_fwd, dict(ldy=63)), (ln_fwd, dict(rows=9)),
    (ln_fwd, dict(rows=-1)), (ln_fwd, dict(h=0)), (ln_fwd, dict(eps=0.0)), (ln_fwd, dict(eps=float("nan"))),
    (ln_fwd, dict(eps=float("inf"))), (ln_fwd, dict(dt=7)), (ln_fwd, dict(wdt=7)), (ln_fwd, dict(idx=P[6], blk=3)),
    (ln_fwd, dict(n=P[6], blk=3)), (ln_fwd, dict(blk=0)), (ln_fwd, dict(idx=P[6], y=P[0])),
    (ln_fwd, dict(y=ctypes.c_void_p((1 << 20) + 256))), (ln_fwd, dict(y=P[0], ldy=128)),
    (ln_fwd, dict(idx=P[6], blk=4, S=10)),
    (ln_bwd, dict(dy=N0)), (ln_bwd, dict(x=N0)), (ln_bwd, dict(mean=N0)), (ln_bwd, dict(rstd=N0)), (ln_bwd, dict(dx=N0)),
    (ln_bwd, dict(ldd=63)), (ln_bwd, dict(dres=P[9], ldr=63)), (ln_bwd, dict(idx=P[9], dx=P[0])),
    (ln_bwd, dict(dx=ctypes.c_void_p((1 << 20) + 16))), (ln_bwd, dict(dres=ctypes.c_void_p((1 << 25) + 16), ldr=64)),
    (lin_fwd, dict(x=N0)), (lin_fwd, dict(w=N0)), (lin_fwd, dict(y=N0)), (lin_fwd, dict(ldx=60)), (lin_fwd, dict(ldx=68)),
    (lin_fwd, dict(ldw=68)), (lin_fwd, dict(x=ctypes.c_void_p((1 << 20) + 8))), (lin_fwd, dict(act=4)),
    (lin_fwd, dict(act=-1)), (lin_fwd, dict(N=0)), (lin_fwd, dict(K=0)), (lin_fwd, dict(M=-1)), (lin_fwd, dict(bdt=5)),
    (lin_fwd, dict(y=P[0])), (lin_fwd, dict(y=P[1])), (lin_fwd, dict(pre=P[3], ldp=64)), (lin_fwd, dict(pre=P[6], ldp=63)),
    (lin_fwd, dict(res=P[3], ldr=72)), (lin_fwd, dict(n=P[6], blk=3)), (lin_fwd, dict(N=1 << 25, ldy=1 << 25)),
    (lin_bwd, dict(dy=N0)), (lin_bwd, dict(pre=N0)), (lin_bwd, dict(x=N0)), (lin_bwd, dict(w=N0)), (lin_bwd, dict(ldp=60)),
    (lin_bwd, dict(ldx=68)), (lin_bwd, dict(ldw=68)), (lin_bwd, dict(dx=P[0])), (lin_bwd, dict(dw=P[1])),
    (lin_bwd, dict(lddw=63)), (lin_bwd, dict(act=9)), (lin_bwd, dict(n=P[8], blk=3)),
    (drop, dict(x=N0)), (drop, dict(y=N0)), (drop, dict(p=-0.1)), (drop, dict(p=1.1)), (drop, dict(p=float("nan"))),
    (drop, dict(cols=0)), (drop, dict(rows=-1)), (drop, dict(ldx=63)), (drop, dict(res=P[2], ldr=63)),
    (drop, dict(row0=-1)), (drop, dict(row0=(1 << 31) - 7)), (drop, dict(idx=P[2], row0=8)),
    (drop, dict(idx=P[2], blk=3)), (drop, dict(y=ctypes.c_void_p((1 << 20) + 16))), (drop, dict(dt=3)),
])
def test_bad_arguments_are_refused(lib, fn, bad):
    assert fn(lib, **bad) == _lib.EINVAL
    assert "jenga_" in _lib.last_error()


def test_sizes_and_workspaces(lib):
    assert ln_fwd(lib, h=16385, ldx=16385, ldy=16385) == _lib.EUNSUPPORTED
    assert ln_bwd(lib, h=16385, ldx=16385, ldy=16385, ldd=16385) == _lib.EUNSUPPORTED
    assert ln_bwd(lib, wsb=16) == _lib.EWORKSPACE and ln_bwd(lib, ws=N0) == _lib.EWORKSPACE
    assert lin_bwd(lib, wsb=16) == _lib.EWORKSPACE and lin_bwd(lib, ws=N0) == _lib.EWORKSPACE
    # nothing to do: no launch, no pointer needed
    assert ln_fwd(lib, rows=0, x=N0, y=N0) == 0 and lin_fwd(lib, M=0, x=N0, y=N0) == 0 and drop(lib, rows=0, x=N0) == 0
    assert lin_bwd(lib, dx=N0, dw=N0, db=N0) == 0
    # the smooth activations keep dz as a pair
    a = lib.jenga_linear_bwd_workspace_bytes(1000, 1544, 520, _lib.ACT_RELU)
    b = lib.jenga_linear_bwd_workspace_bytes(1000, 1544, 520, _lib.ACT_GELU)
    assert a >= 1000 * 1544 * 2 and b - a >= 1000 * 1544 * 2
    assert lib.jenga_layernorm_bwd_workspace_bytes(1, 4096) >= 8 * 4096


def test_binding_refuses_cpu_tensors():
    import token_sparse_long_b200 as J
    x = torch.zeros(4, 64)
    for call in (lambda: J.jenga_layernorm_fwd(x), lambda: J.jenga_linear_fwd(x.bfloat16(), x.bfloat16()),
                 lambda: J.jenga_dropout(x, 0.1, 1)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
