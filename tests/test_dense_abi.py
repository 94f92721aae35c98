"""Host-side checks of the dense operators (no GPU): shapes of launches and refusals before any."""
import ctypes

import numpy as np
import pytest

from token_sparse_long_b200 import _lib


@pytest.fixture(scope="module")
def lib():
    from token_sparse_long_b200 import build
    build.build()
    return _lib.load()


def test_rows_pass_stage_belongs_to_one_group(lib):
    # 8 / G groups of G warps take the rows of w in turn, row i from stage i % stages: only with a
    # whole number of stages per group is a stage always the same group's
    for M in (1, 2):
        for K in range(8, 16385, 8):
            g, s = ctypes.c_int(), ctypes.c_int()
            assert lib.jenga_test_linear_rows_shape(M, K, ctypes.byref(g), ctypes.byref(s)) == 0
            groups = 8 // g.value
            assert g.value in (1, 2, 4, 8) and s.value >= groups and s.value % groups == 0, (M, K, g.value, s.value)
            assert s.value <= 64 and s.value * K * 2 <= 192 * 1024
    assert lib.jenga_test_linear_rows_shape(3, 64, ctypes.byref(g), ctypes.byref(s)) == _lib.EINVAL


# Addresses below are never read: every call ends on the host.
BASE, MB = 1 << 40, 1 << 20


def at(mb):
    return ctypes.c_void_p(BASE + mb * MB)


def lin_fwd(lib, **k):
    a = dict(x=at(0), ldx=512, w=at(1), ldw=512, bias=at(2), bdt=_lib.F32, act=0, res=at(3), ldr=256, M=64, N=256, K=512,
             nk=None, blk=1, y=at(4), ldy=256, pre=at(5), ldp=256, ws=None, nws=0)
    a.update(k)
    return lib.jenga_linear_fwd(*[a[n] for n in "x ldx w ldw bias bdt act res ldr M N K nk blk y ldy pre ldp ws nws".split()],
                                None)


def lin_bwd(lib, **k):
    a = dict(dy=at(0), ldy=256, x=at(1), ldx=512, w=at(2), ldw=512, act=1, pre=at(3), ldp=256, M=64, N=256, K=512, nk=None,
             blk=1, dx=at(4), ldd=512, dw=at(5), lddw=512, db=at(6), acc=0, ws=None, nws=0)
    a.update(k)
    return lib.jenga_linear_bwd(*[a[n] for n in "dy ldy x ldx w ldw act pre ldp M N K nk blk dx ldd dw lddw db acc ws "
                                  "nws".split()], None)


def ln_fwd(lib, **k):
    a = dict(x=at(0), ldx=256, S=64, h=256, idx=None, nk=None, blk=1, rows=64, ga=at(1), be=at(2), wdt=_lib.F32, eps=1e-5,
             dt=_lib.BF16, y=at(3), ldy=256, mean=at(4), rstd=at(5))
    a.update(k)
    return lib.jenga_layernorm_fwd(*[a[n] for n in "x ldx S h idx nk blk rows ga be wdt eps dt y ldy mean rstd".split()], None)


def ln_bwd(lib, **k):
    a = dict(dy=at(0), ldy=256, x=at(1), ldx=256, S=64, h=256, idx=None, nk=None, blk=1, rows=64, mean=at(2), rstd=at(3),
             ga=at(4), wdt=_lib.F32, dres=at(5), ldr=256, dt=_lib.BF16, dx=at(6), ldd=256, dg=at(7), db=at(8), acc=0,
             ws=None, nws=0)
    a.update(k)
    return lib.jenga_layernorm_bwd(*[a[n] for n in "dy ldy x ldx S h idx nk blk rows mean rstd ga wdt dres ldr dt dx ldd dg "
                                     "db acc ws nws".split()], None)


def off(mb, nbytes):
    return ctypes.c_void_p(BASE + mb * MB + nbytes)


def test_outputs_that_meet_an_input_or_each_other_are_refused(lib):
    # what the backward calls get when nothing meets: the missing workspace ends them
    assert lin_bwd(lib) == _lib.EWORKSPACE and ln_bwd(lib) == _lib.EWORKSPACE
    for k in (dict(db=off(0, 64 * 512 - 4)), dict(db=off(1, 0)), dict(db=off(2, 4096)), dict(db=off(3, 0)), dict(db=off(4, 0)),
              dict(db=off(5, 2048)), dict(dx=off(5, 0)), dict(dw=off(4, 1024)), dict(nk=at(6)), dict(dx=at(1)), dict(dx=at(0))):
        assert lin_bwd(lib, **k) == _lib.EINVAL, k
    need = lib.jenga_linear_bwd_workspace_bytes(64, 256, 512, 1)
    for mb in range(7):
        assert lin_bwd(lib, ws=off(mb, 0), nws=need) == _lib.EINVAL, mb
    for k in (dict(y=at(2), ldy=256), dict(pre=off(2, 1020)), dict(y=at(5)), dict(y=at(3), ldy=264), dict(nk=at(4)),
              dict(y=off(0, 1024), ldy=256)):
        assert lin_fwd(lib, **k) == _lib.EINVAL, k
    for k in (dict(y=at(1)), dict(mean=off(0, 256)), dict(rstd=at(4)), dict(mean=off(5, 252)), dict(y=off(2, 16)),
              dict(rstd=off(3, 64 * 512 - 4)), dict(idx=at(3), blk=32), dict(nk=at(4)), dict(y=at(0), idx=at(9), blk=32)):
        assert ln_fwd(lib, **k) == _lib.EINVAL, k
    for k in (dict(dg=at(4)), dict(dg=at(8)), dict(db=off(0, 0)), dict(dx=at(2)), dict(dx=off(3, 252)), dict(db=at(6)),
              dict(dx=at(6), nk=off(6, 512 * 63)), dict(dx=off(1, 512)), dict(dx=at(0), idx=at(9), blk=32)):
        assert ln_bwd(lib, **k) == _lib.EINVAL, k
    need = lib.jenga_layernorm_bwd_workspace_bytes(64, 256)
    for mb in range(9):
        assert ln_bwd(lib, ws=off(mb, 0), nws=need) == _lib.EINVAL, mb
    drop = lambda **k: lib.jenga_dropout(*[{**dict(x=at(0), ldx=64, r=at(1), ldr=64, rows=64, cols=64, idx=None, nk=None, blk=32,
                                                   row0=0, p=0.5, seed=1, off=2, dt=_lib.BF16, y=at(2), ldy=64), **k}[n]
                                           for n in "x ldx r ldr rows cols idx nk blk row0 p seed off dt y ldy".split()], None)
    for k in (dict(y=off(0, 128)), dict(y=at(1), ldy=72), dict(idx=off(2, 8)), dict(nk=off(2, 64 * 128 - 4))):
        assert drop(**k) == _lib.EINVAL, k


def test_the_same_matrix_and_columns_side_by_side_are_no_overlap(lib):
    # allowed in place: dx on dres, x or dy
    for k in (dict(dx=at(5)), dict(dx=at(1)), dict(dx=at(0)), dict(dx=at(5), x=at(5))):
        assert ln_bwd(lib, **k) == _lib.EWORKSPACE, k
    # columns of one matrix: x and dx halves of rows of 1024, dy, pre thirds of rows of 768, one row in a gap
    assert lin_bwd(lib, x=at(1), ldx=1024, dx=off(1, 1024), ldd=1024) == _lib.EWORKSPACE
    assert lin_bwd(lib, x=off(1, 1024), ldx=1024, dx=at(1), ldd=1024) == _lib.EWORKSPACE
    assert lin_bwd(lib, x=at(1), ldx=1024, dx=off(1, 1022), ldd=1024) == _lib.EINVAL
    assert lin_bwd(lib, x=at(1), ldx=1024, dx=off(1, 1026), ldd=1024) == _lib.EINVAL
    assert lin_bwd(lib, x=at(1), ldx=1024, dx=off(1, 1024), ldd=1032) == _lib.EINVAL
    assert ln_bwd(lib, dy=at(0), ldy=768, dres=off(0, 512), ldr=768, dx=off(0, 1024), ldd=768) == _lib.EWORKSPACE
    assert ln_bwd(lib, x=at(1), ldx=512, dg=off(1, 512), h=128, ldy=128, ldr=128, ldd=128) == _lib.EWORKSPACE
    assert ln_bwd(lib, x=at(1), ldx=512, dg=off(1, 516 + 256), h=128, ldy=128, ldr=128, ldd=128) == _lib.EINVAL


def test_a_single_row_has_no_pitch(lib):
    one = dict(M=1, K=521, ldx=521, ldw=528, dx=None, pre=at(3), lddw=521)
    assert lin_bwd(lib, **one) == _lib.EWORKSPACE
    assert lin_bwd(lib, M=64, N=1, K=521, ldx=528, ldw=521, ldd=521, lddw=521) == _lib.EWORKSPACE
    assert lin_bwd(lib, **{**one, "M": 2}) == _lib.EINVAL  # two rows: the second is not 16-byte aligned
    assert lin_bwd(lib, **{**one, "x": off(1, 2)}) == _lib.EINVAL
    need = lib.jenga_linear_fwd_workspace_bytes(1, 256, 8193)  # split reduction: ends at the missing workspace
    assert need > 0 and lin_fwd(lib, M=1, K=8193, ldx=8193, ldw=8200, w=at(16)) == _lib.EWORKSPACE
    assert lin_fwd(lib, M=2, K=8193, ldx=8193, ldw=8200, w=at(16)) == _lib.EINVAL


def test_oracle_relu_keeps_nan():
    from oracle import dense as od
    y = od.act(np.array([-1.0, 0.0, 2.0, np.nan, -np.inf, np.inf]), "relu")
    assert np.array_equal(y, [0.0, 0.0, 2.0, np.nan, 0.0, np.inf], equal_nan=True)


def test_workspace_of_sizes_that_are_refused(lib):
    big = 2 ** 31 - 1
    for M, N, K in ((big, 8, 8), (2 ** 30 + 1, 8, 8), (8, big, 8), (8, 8, big), (8, 2 ** 24 + 1, 8), (0, 8, 8), (8, -1, 8)):
        assert lib.jenga_linear_fwd_workspace_bytes(M, N, K) == 0 and lib.jenga_linear_bwd_workspace_bytes(M, N, K, 2) == 0
        assert lin_fwd(lib, M=M, N=N, K=K, ldx=K, ldw=K, ldr=N, ldy=N, ldp=N) in (0 if M == 0 else _lib.EINVAL, _lib.EINVAL)
    assert lib.jenga_linear_bwd_workspace_bytes(2 ** 30, 8, 8, 2) >= 3 * 2 * 2 ** 30 * 64
    assert lib.jenga_layernorm_bwd_workspace_bytes(big, 8) > 0 and lib.jenga_layernorm_bwd_workspace_bytes(big, 16385) == 0


def test_binding_refuses_what_an_int_does_not_hold():
    import torch
    from token_sparse_long_b200 import api
    m = lambda *s: torch.empty(*s, device="meta", dtype=torch.bfloat16)
    big = 2 ** 31 - 1
    assert api._mat(m(big, 1), "x") == 1 and api._mat(m(2, big), "x") == big
    for shape in ((2 ** 31, 1), (2 ** 32 + 5, 1), (1, 2 ** 31), (2, 2 ** 32 + 8)):
        with pytest.raises(ValueError):
            api._mat(m(*shape), "x")
    idx = torch.zeros(4096, dtype=torch.int32)
    assert api._rows_arg(idx, None, 2 ** 19 - 1, None, 0) == 4096 * (2 ** 19 - 1)
    assert api._rows_arg(None, None, 32, None, 640) == 640
    for blk in (2 ** 20, 2 ** 32 + 32, 0, -1):
        with pytest.raises(ValueError):
            api._rows_arg(idx, None, blk, None, 0)


def test_linear_bwd_workspace_without_dw(lib):
    size = lambda act: lib.jenga_linear_bwd_workspace_bytes(26240, 11008, 4096, act)
    assert size(2) - size(1) >= 2 * 2 * 26240 * 11008  # two more bf16 parts of dz, for dw alone
    for act in (2, 3):
        # the size is checked before the overlap: one byte short and then a workspace on dy
        small = lib.jenga_linear_bwd_workspace_bytes(64, 256, 512, 1)
        k = dict(act=act, dw=None, ws=at(0))
        assert lin_bwd(lib, nws=small - 1, **k) == _lib.EWORKSPACE and lin_bwd(lib, nws=small, **k) == _lib.EINVAL
        k["dw"] = at(5)
        assert lin_bwd(lib, nws=small, **k) == _lib.EWORKSPACE
