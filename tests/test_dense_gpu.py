"""GPU parity of layer norm, linear layer and dropout (forward and backward) against the float64
oracle.  Bars follow from the arithmetic: u = 2^-24 is half an fp32 step and RB = 2^-8 half a
bf16 step, relative to the value; a sum of n fp32 terms is off by at most n u times the sum of
magnitudes (2 n u on the tensor core, which truncates)."""
import numpy as np
import pytest
import torch

from oracle import dense as od

pytestmark = pytest.mark.gpu

U, RB = 2.0 ** -24, 2.0 ** -8
HALF = {torch.float32: U, torch.bfloat16: RB}
NAN = float("nan")


@pytest.fixture(scope="module")
def J():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import token_sparse_long_b200 as J
    J._lib.load()
    return J


def f64(t):
    return t.detach().double().cpu().numpy()


def randn(seed, *shape, dt=torch.float32, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale + shift).to(dt).cuda()


def pitched(t, extra):
    """The same matrix with `extra` more elements between rows (NaN)."""
    b = torch.full((t.shape[0], t.shape[1] + extra), NAN, dtype=t.dtype, device=t.device)
    b[:, :t.shape[1]] = t
    return b[:, :t.shape[1]]


def close(got, want, tol):
    got = f64(got)
    assert got.shape == want.shape
    err = np.abs(got - want)
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), float(np.nanmax(err / tol)), np.argwhere(bad)[:4].tolist())


# ------------------------------------------------------------------ layer norm
def ln_tol(x, mean, rstd, gamma, y, dt):
    """|y - exact|: a row's sums run over at most h / 32 + 40 sequential adds; the mean is off by
    that many u of mean|x|, n by the mean's error and a few relative errors of var and rstd."""
    h = x.shape[1]
    k = h / 32 + 40
    dm = k * U * np.abs(x).mean(1)
    n = np.abs(x - mean[:, None]) * rstd[:, None]
    rel = (k + 8) * U + 2 * dm * rstd
    dn = n * rel[:, None] + (dm * rstd)[:, None] + 4 * U * n
    return dn * np.abs(gamma) * 1.01 + 4 * U * (n * np.abs(gamma) + np.abs(y)) + HALF[dt] * np.abs(y) + 1e-30


LN_SIZES = [(1, 1), (3, 7), (5, 64), (130, 256), (257, 1000), (64, 1001), (33, 4096), (9, 5120), (3, 8192), (4, 16384),
            (3, 16383), (300, 40)]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,h", LN_SIZES)
def test_layernorm_fwd(J, rows, h, dt):
    for wdt in (torch.float32, torch.bfloat16):
        x = randn(h, rows, h, dt=dt, scale=2.0, shift=10.0)
        ga, be = randn(1, h, dt=wdt, scale=0.3, shift=1.0), randn(2, h, dt=wdt)
        y, mean, rstd = J.jenga_layernorm_fwd(x, ga, be)
        J.jenga_check_device_status()
        ry, rm, rr = od.layernorm_fwd(f64(x), f64(ga), f64(be))
        tol = ln_tol(f64(x), rm, rr, f64(ga), ry, dt)
        close(y, ry, tol + 4 * U * np.abs(f64(be)))
        k = h / 32 + 40
        close(mean, rm, (k + 2) * U * np.abs(f64(x)).mean(1) + 1e-30)
        close(rstd, rr, rr * ((k + 10) * U + 2 * k * U * np.abs(f64(x)).mean(1) * rr))


def test_layernorm_fwd_without_parameters_pitched_and_in_place(J):
    x = randn(3, 70, 512, dt=torch.bfloat16)
    want = J.jenga_layernorm_fwd(x)[0]
    close(want, od.layernorm_fwd(f64(x))[0], ln_tol(f64(x), *od.layernorm_fwd(f64(x))[1:], np.ones(512),
                                                      od.layernorm_fwd(f64(x))[0], torch.bfloat16))
    for extra in (8, 3):  # 16-byte rows, unaligned rows
        out = pitched(torch.zeros_like(x), 5)
        assert torch.equal(J.jenga_layernorm_fwd(pitched(x, extra), out=out)[0], want) or extra == 3
        close(out, f64(want), RB * 2 * np.abs(f64(want)) + 1e-6)
        assert torch.isnan(out._base[:, 512:]).all()
    y = x.clone()
    J.jenga_layernorm_fwd(y, out=y)
    assert torch.equal(y, want)


def test_layernorm_row_far_off_zero(J):
    # mean 1000 times the spread: a one-pass sum of squares would lose every digit
    x = randn(4, 8, 1024, scale=1.0, shift=1000.0)
    y, mean, rstd = J.jenga_layernorm_fwd(x)
    ry, rm, rr = od.layernorm_fwd(f64(x))
    close(y, ry, ln_tol(f64(x), rm, rr, np.ones(1024), ry, torch.float32))
    assert np.abs(f64(rstd) / rr - 1).max() < 1e-5


def kept(S, blk, n, seed):
    idx = torch.randperm(S // blk, generator=torch.Generator().manual_seed(seed))[:n].sort().values.to(torch.int32)
    rows = (idx.long()[:, None] * blk + torch.arange(blk)[None, :]).reshape(-1)
    return idx.cuda(), rows.cuda()


@pytest.mark.parametrize("h", [256, 1001])
def test_layernorm_through_the_block_list(J, h):
    S, blk, n, cap = 512, 32, 7, 11
    x = randn(5, S, h, dt=torch.bfloat16)
    idx, rows = kept(S, blk, n, 6)
    mask = torch.ones(S, dtype=torch.bool, device="cuda")
    mask[rows] = False
    x[mask] = NAN  # eliminated rows are never read
    lst = torch.full((cap,), -1, dtype=torch.int32, device="cuda")
    lst[:n] = idx
    nk = torch.tensor([n], dtype=torch.int32, device="cuda")
    ga, be = randn(7, h, dt=torch.bfloat16), randn(8, h, dt=torch.bfloat16)
    out = torch.full((cap * blk, h), 7.0, dtype=torch.bfloat16, device="cuda")
    y, mean, rstd = J.jenga_layernorm_fwd(x, ga, be, idx=lst, n_kept=nk, blk=blk, out=out)
    want, wm, wr = J.jenga_layernorm_fwd(x[rows].contiguous(), ga, be)
    assert torch.equal(y[:n * blk], want) and torch.equal(mean[:n * blk], wm) and torch.equal(rstd[:n * blk], wr)
    assert (y[n * blk:] == 7.0).all()  # rows behind the count stay as they were
    # backward: dx lands on the same sequence rows, the others keep the residual gradient
    dy = randn(9, cap * blk, h, dt=torch.bfloat16)
    dy[n * blk:] = NAN
    G = randn(10, S, h, dt=torch.bfloat16)
    dx = G.clone()
    _, dg, db = J.jenga_layernorm_bwd(dy, x, mean, rstd, ga, idx=lst, n_kept=nk, blk=blk, dres=dx, dx=dx)
    J.jenga_check_device_status()
    w = J.jenga_layernorm_bwd(dy[:n * blk], x[rows].contiguous(), wm, wr, ga, dres=G[rows].contiguous())
    assert torch.equal(dx[rows], w[0]) and torch.equal(dx[mask], G[mask])
    k = n * blk * U * 3
    xh = (f64(x[rows]) - f64(wm)[:, None]) * f64(wr)[:, None]
    close(dg, f64(w[1]), k * np.abs(f64(dy[:n * blk]) * xh).sum(0) + 1e-30)
    close(db, f64(w[2]), k * np.abs(f64(dy[:n * blk])).sum(0) + 1e-30)
    # no block kept: nothing written, empty sums
    nk.zero_()
    y2 = out.clone()
    J.jenga_layernorm_fwd(x, ga, be, idx=lst, n_kept=nk, blk=blk, out=y2)
    assert torch.equal(y2, out)
    _, dg, db = J.jenga_layernorm_bwd(dy, x, mean, rstd, ga, idx=lst, n_kept=nk, blk=blk, dx=dx)
    assert not dg.any() and not db.any()


@pytest.mark.parametrize("entries", [[3, 99, 5], [3, -1, 5], [3, 3, 5], [5, 3, 7]])
def test_bad_list_entries_are_recorded_and_skipped(J, entries):
    S, blk, h = 512, 32, 256
    x = randn(11, S, h)
    lst = torch.tensor(entries, dtype=torch.int32, device="cuda")
    out = torch.full((3 * blk, h), 7.0, device="cuda")
    J.jenga_layernorm_fwd(x, idx=lst, blk=blk, out=out)
    with pytest.raises(J._lib.JengaError) as e:
        J.jenga_check_device_status()
    assert e.value.status == J._lib.EINTERNAL
    assert (out[blk:2 * blk] == 7.0).all() and not (out[:blk] == 7.0).all()
    # the third entry is fine unless it fails to ascend past the second
    assert bool((out[2 * blk:] == 7.0).all()) == (entries[2] <= entries[1])
    dx = torch.zeros(S, h, device="cuda")
    st = torch.ones(3 * blk, device="cuda")
    J.jenga_layernorm_bwd(out, x, st, st, idx=lst, blk=blk, dx=dx)
    with pytest.raises(J._lib.JengaError):
        J.jenga_check_device_status()
    y = torch.full((3 * blk, h), 7.0, device="cuda")
    J.jenga_dropout(out, 0.5, 1, idx=torch.tensor([3, -2, 5], dtype=torch.int32, device="cuda"), blk=blk, out=y)
    with pytest.raises(J._lib.JengaError):
        J.jenga_check_device_status()
    assert (y[blk:2 * blk] == 7.0).all()


def test_count_out_of_range_is_recorded(J):
    x = randn(12, 64, 256, dt=torch.bfloat16)
    w = randn(13, 64, 256, dt=torch.bfloat16)
    for bad in (3, -1):
        nk = torch.tensor([bad], dtype=torch.int32, device="cuda")
        for call in (lambda: J.jenga_layernorm_fwd(x, n_kept=nk, blk=32), lambda: J.jenga_dropout(x, 0.5, 1, n_kept=nk, blk=32),
                     lambda: J.jenga_linear_fwd(x, w, n_kept=nk, blk=32)):
            call()
            with pytest.raises(J._lib.JengaError) as e:
                J.jenga_check_device_status()
            assert e.value.status == J._lib.EINTERNAL


@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,h", LN_SIZES + [(2000, 96)])
def test_layernorm_bwd(J, rows, h, dt, res):
    x, dy = randn(h, rows, h, dt=dt, scale=2.0, shift=3.0), randn(h + 1, rows, h, dt=dt)
    ga = randn(1, h, dt=dt, scale=0.3, shift=1.0)
    dres = randn(2, rows, h, dt=dt) if res else None
    _, mean, rstd = J.jenga_layernorm_fwd(x, ga)
    dx, dg, db = J.jenga_layernorm_bwd(dy, x, mean, rstd, ga, dres=dres)
    J.jenga_check_device_status()
    X, D, GA, m, r = (f64(t) for t in (x, dy, ga, mean, rstd))
    wx, wg, wb = od.layernorm_bwd(D, X, m, r, GA)
    if res:
        wx = wx + f64(dres)
    n = np.abs((X - m[:, None]) * r[:, None])
    g = np.abs(D * GA)
    k = h / 32 + 60
    c1, c2 = g.mean(1, keepdims=True), (g * n).mean(1, keepdims=True)
    tol = r[:, None] * (6 * U * g + (k + 6) * U * c1 + n * (k + 12) * U * c2) + HALF[dt] * np.abs(wx) + 4 * U * np.abs(wx)
    if res:
        tol = tol + 2 * U * np.abs(f64(dres))
    close(dx, wx, tol * 1.01 + 1e-30)
    close(dg, wg, (rows + 10) * U * (np.abs(D) * n).sum(0) + 1e-30)
    close(db, wb, (rows + 10) * U * np.abs(D).sum(0) + 1e-30)
    # accumulate, and a second run gives the same bits
    dg2, db2 = torch.ones_like(dg), torch.full_like(db, -2.0)
    J.jenga_layernorm_bwd(dy, x, mean, rstd, ga, dres=dres, dgamma=dg2, dbeta=db2, accumulate=True)
    assert torch.equal(dg2, dg + 1.0) and torch.equal(db2, db - 2.0)
    dx3, none_g, none_b = J.jenga_layernorm_bwd(dy, x, mean, rstd, ga, dres=dres, weight_grads=False)
    assert torch.equal(dx3, dx) and none_g is None and none_b is None


@pytest.mark.parametrize("rows,h,dt", [(5000, 4096, torch.bfloat16), (3200, 5120, torch.bfloat16),
                                       (4000, 2048, torch.float32), (20000, 264, torch.bfloat16)])
def test_layernorm_many_rows_a_group(J, rows, h, dt):
    """More rows a group than the ring has stages, through a list with a bad entry in the middle."""
    blk = 40
    S = rows + 5 * blk
    x = randn(h, S, h, dt=dt, shift=1.0)
    ga, be = randn(1, h, dt=dt, shift=1.0), randn(2, h, dt=dt)
    lst, rowsel = kept(S, blk, rows // blk, 3)
    bad = rows // blk // 2
    ok = torch.ones(rows, dtype=torch.bool, device="cuda")
    want = J.jenga_layernorm_fwd(x[rowsel].contiguous(), ga, be)
    ry, rm, rr = od.layernorm_fwd(f64(x[rowsel]), f64(ga), f64(be))
    close(want[0], ry, ln_tol(f64(x[rowsel]), rm, rr, f64(ga), ry, dt) + 4 * U * np.abs(f64(be)))
    for spoil in (False, True):
        if spoil:
            lst[bad] = S
            ok[bad * blk:(bad + 2) * blk] = False  # the entry, and the next one, which is not above it
        y, mean, rstd = J.jenga_layernorm_fwd(x, ga, be, idx=lst, blk=blk, out=torch.full((rows, h), 7.0, dtype=dt, device="cuda"))
        assert torch.equal(y[ok], want[0][ok]) and torch.equal(mean[ok], want[1][ok])
        assert (y[~ok] == 7.0).all()
        mean[~ok], rstd[~ok] = 0.0, 1.0
        dy = randn(4, rows, h, dt=dt)
        dx, dg, db = J.jenga_layernorm_bwd(dy, x, mean, rstd, ga, idx=lst, blk=blk)
        if spoil:
            with pytest.raises(J._lib.JengaError):
                J.jenga_check_device_status()
        else:
            J.jenga_check_device_status()
        k = ok.cpu().numpy()
        X, D = f64(x[rowsel])[k], f64(dy)[k]
        m, r = f64(mean)[k], f64(rstd)[k]
        wx, wg, wb = od.layernorm_bwd(D, X, m, r, f64(ga))
        n = np.abs((X - m[:, None]) * r[:, None])
        g = np.abs(D * f64(ga))
        q = h / 32 + 60
        c1, c2 = g.mean(1, keepdims=True), (g * n).mean(1, keepdims=True)
        tol = r[:, None] * (6 * U * g + (q + 6) * U * c1 + n * (q + 12) * U * c2) + (HALF[dt] + 4 * U) * np.abs(wx)
        close(dx[rowsel][ok], wx, tol * 1.01 + 1e-30)
        close(dg, wg, (rows + 10) * U * (np.abs(D) * n).sum(0) + 1e-30)
        close(db, wb, (rows + 10) * U * np.abs(D).sum(0) + 1e-30)


@pytest.mark.parametrize("h,res", [(16384, False), (16384, True), (12288, True), (14000, False), (9216, True)])
def test_layernorm_bwd_rows_that_fill_the_ring(J, h, res):
    """fp32 rows of which shared memory holds one or two at a time, several a CTA, through a list
    with a bad entry."""
    blk, rows, dt = 8, 640, torch.float32
    S = rows + 9 * blk
    x = randn(h, S, h, dt=dt, shift=1.0)
    ga = randn(1, h, dt=dt, shift=1.0)
    lst, rowsel = kept(S, blk, rows // blk, 3)
    dres = randn(5, S, h, dt=dt) if res else None
    _, mean, rstd = J.jenga_layernorm_fwd(x, ga, ga, idx=lst, blk=blk)
    dy = randn(4, rows, h, dt=dt)
    bad = rows // blk // 2
    ok = torch.ones(rows, dtype=torch.bool, device="cuda")
    for spoil in (False, True):
        if spoil:
            lst[bad] = S
            ok[bad * blk:(bad + 2) * blk] = False  # the entry, and the next one, which is not above it
        out = torch.full((S, h), 7.0, dtype=dt, device="cuda")
        dx, dg, db = J.jenga_layernorm_bwd(dy, x, mean, rstd, ga, idx=lst, blk=blk, dres=dres, dx=out)
        if spoil:
            with pytest.raises(J._lib.JengaError):
                J.jenga_check_device_status()
        else:
            J.jenga_check_device_status()
        other = torch.ones(S, dtype=torch.bool, device="cuda")
        other[rowsel[ok]] = False
        assert (dx[other] == 7.0).all()
        sel = rowsel[ok]
        X, D, m, r = f64(x[sel]), f64(dy[ok]), f64(mean[ok]), f64(rstd[ok])
        wx, wg, wb = od.layernorm_bwd(D, X, m, r, f64(ga))
        n = np.abs((X - m[:, None]) * r[:, None])
        g = np.abs(D * f64(ga))
        q = h / 32 + 60
        c1, c2 = g.mean(1, keepdims=True), (g * n).mean(1, keepdims=True)
        tol = r[:, None] * (6 * U * g + (q + 6) * U * c1 + n * (q + 12) * U * c2)
        if res:
            E = f64(dres[sel])
            wx, tol = wx + E, tol + 2 * U * np.abs(E)
        tol = tol + (HALF[dt] + 4 * U) * np.abs(wx)
        close(dx[sel], wx, tol * 1.01 + 1e-30)
        close(dg, wg, (rows + 10) * U * (np.abs(D) * n).sum(0) + 1e-30)
        close(db, wb, (rows + 10) * U * np.abs(D).sum(0) + 1e-30)


def test_layernorm_unaligned_bases_and_in_place_gradients(J):
    bf = torch.bfloat16
    x, dy = randn(1, 90, 520, dt=bf), randn(2, 90, 520, dt=bf)
    ga, be = randn(3, 520, dt=bf, shift=1.0), randn(4, 520, dt=bf)
    y, mean, rstd = J.jenga_layernorm_fwd(x, ga, be)
    wx, wg, wb = J.jenga_layernorm_bwd(dy, x, mean, rstd, ga)

    def off(t):  # the same values one element into a buffer
        b = torch.full((t.numel() + 1,), NAN, dtype=t.dtype, device="cuda")
        b[1:] = t.reshape(-1)
        return b[1:].view(t.shape)

    y2, m2, r2 = J.jenga_layernorm_fwd(off(x), off(ga), be)
    close(y2, f64(y), 2 * RB * np.abs(f64(y)) + 1e-6)
    x2, g2, b2 = J.jenga_layernorm_bwd(off(dy), x, mean, rstd, off(ga))
    close(x2, f64(wx), 2 * RB * np.abs(f64(wx)) + 1e-6)
    close(g2, f64(wg), 1e-5 * np.abs(f64(wg)) + 1e-4)
    for which in ("dy", "x"):
        a, b = dy.clone(), x.clone()
        out = a if which == "dy" else b
        J.jenga_layernorm_bwd(a, b, mean, rstd, ga, dx=out)
        assert torch.equal(out, wx)
    nx = J.jenga_layernorm_bwd(dy, x, mean, rstd)[0]
    rx, _, _ = od.layernorm_bwd(f64(dy), f64(x), f64(mean), f64(rstd))
    close(nx, rx, RB * np.abs(rx) * 1.01 + 1e-4 * f64(rstd)[:, None])
    J.jenga_check_device_status()


# ------------------------------------------------------------------ linear
ACTS = ["none", "relu", "gelu", "silu"]


def act_err(z, kind):
    """Error of the activation's own evaluation: erff is within 2 ulp of a value up to 1, __expf
    within 2 + 1.173 |z| ulp, each division or product within 2 ulp."""
    a = np.abs(z)
    return {"none": 0.0, "relu": 0.0, "gelu": 6 * 2 * U * a, "silu": (8 + 1.2 * a) * 2 * U * a}[kind] + 1e-30


def lin_case(M, N, K, bdt=torch.float32):
    x = randn(M + K, M, (K + 7) // 8 * 8, dt=torch.bfloat16)[:, :K]  # 16-byte aligned rows for any K
    w = randn(N + K + 1, N, (K + 7) // 8 * 8, dt=torch.bfloat16, scale=1.5 / K ** 0.5)[:, :K]
    return x, w, randn(3, N, dt=bdt, scale=0.5), randn(4, M, N, dt=torch.bfloat16)


LIN_SIZES = [(1, 1, 1), (1, 64, 64), (1, 1541, 520), (2, 512, 4096), (7, 33, 72), (15, 300, 1000), (17, 96, 200),
             (33, 700, 64), (64, 256, 2048), (100, 129, 130), (128, 128, 64), (257, 300, 1001), (300, 1541, 520),
             (600, 512, 256), (1100, 260, 136), (2500, 2304, 192)]


@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("M,N,K", LIN_SIZES)
def test_linear_fwd(J, M, N, K, kind):
    for bdt, with_res, with_pre in ((torch.float32, True, True), (torch.bfloat16, False, False), (None, True, False)):
        x, w, b, res = lin_case(M, N, K, bdt or torch.float32)
        bias, residual = b if bdt else None, res if with_res else None
        y, pre = J.jenga_linear_fwd(x, w, bias, act=kind, residual=residual, save_pre=with_pre)
        J.jenga_check_device_status()
        B = f64(bias) if bdt else None
        ry, rz = od.linear_fwd(f64(x), f64(w), B, kind, f64(res) if with_res else None)
        S = np.abs(f64(x)) @ np.abs(f64(w)).T + (np.abs(B) if bdt else 0.0)
        ez = 2 * (K + 2) * U * S  # |activation slope| <= 1.13
        close(y, ry, 1.13 * ez + act_err(rz, kind) + 4 * U * np.abs(ry) + RB * np.abs(ry) * 1.001
              + (2 * U * np.abs(f64(res)) if with_res else 0.0))
        if with_pre:
            close(pre, rz, ez + RB * np.abs(rz) * 1.001 + 1e-30)


def test_linear_fwd_pitches_and_in_place_residual(J):
    x, w, b, res = lin_case(77, 200, 96)
    want, _ = J.jenga_linear_fwd(x, w, b, act="relu", residual=res)
    for extra in (8, 3):
        out, pre = pitched(torch.zeros_like(res), extra), pitched(torch.zeros_like(res), extra)
        got, _ = J.jenga_linear_fwd(pitched(x, 8), pitched(w, 16), b, act="relu", residual=pitched(res, extra), out=out,
                                    pre=pre)
        assert torch.equal(got, want)
        assert torch.isnan(out._base[:, 200:]).all() and torch.isnan(pre._base[:, 200:]).all()
    y = res.clone()
    J.jenga_linear_fwd(x, w, b, act="relu", residual=y, out=y)
    assert torch.equal(y, want)


@pytest.mark.parametrize("M", [4, 96, 640])
def test_linear_fwd_device_count(J, M):
    blk = M // 4 if M == 4 else 32
    x, w, b, res = lin_case(M, 300, 264)
    want, wpre = J.jenga_linear_fwd(x, w, b, act="gelu", residual=res, save_pre=True)
    for n in (0, 1, M // blk - 1, M // blk):
        v = n * blk
        x2 = x.clone()
        x2[v:] = NAN
        out, pre = (torch.full((M, 300), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        J.jenga_linear_fwd(x2, w, b, act="gelu", residual=res, n_kept=torch.tensor([n], dtype=torch.int32, device="cuda"),
                           blk=blk, out=out, pre=pre)
        J.jenga_check_device_status()
        assert torch.equal(out[:v], want[:v]) and torch.equal(pre[:v], wpre[:v])
        assert (out[v:] == 7.0).all() and (pre[v:] == 7.0).all()


@pytest.mark.parametrize("M,N,K", [(1, 700, 512), (2, 300, 4096), (20, 520, 4096), (96, 300, 4096), (300, 260, 2048),
                                   (3000, 3, 70), (1500, 1100, 64)])
def test_linear_fwd_every_shape_in_place_and_counted(J, M, N, K):
    """Each route (rows of w, swapped, split reductions, wide) with y = residual and a device count."""
    x, w, b, res = lin_case(M, N, K)
    want, wpre = J.jenga_linear_fwd(x, w, b, act="silu", residual=res, save_pre=True)
    ry, rz = od.linear_fwd(f64(x), f64(w), f64(b), "silu", f64(res))
    S = np.abs(f64(x)) @ np.abs(f64(w)).T + np.abs(f64(b))
    close(want, ry, 1.13 * 2 * (K + 2) * U * S + act_err(rz, "silu") + (4 * U + RB * 1.001) * np.abs(ry)
          + 2 * U * np.abs(f64(res)))
    y = res.clone()
    J.jenga_linear_fwd(x, w, b, act="silu", residual=y, out=y)
    assert torch.equal(y, want)
    n = M // 2
    x2, y2 = pitched(x, -K % 8 + 8), res.clone()
    x2[n:] = NAN
    J.jenga_linear_fwd(x2, w, b, act="silu", residual=y2, out=y2, n_kept=torch.tensor([n], dtype=torch.int32, device="cuda"))
    assert torch.equal(y2[:n], want[:n]) and torch.equal(y2[n:], res[n:])
    J.jenga_check_device_status()


def test_linear_bwd_split_sum_with_a_device_count(J):
    M, N, K = 2560, 300, 136  # dw's reduction is split over idle SM pairs
    x, w, _, dy = lin_case(M, N, K)
    pre = randn(9, M, N, dt=torch.bfloat16)
    for v in (0, 65, 1300, M):
        x2, dy2 = x.clone(), dy.clone()
        x2[v:], dy2[v:] = NAN, NAN
        dw = pitched(torch.ones(N, K, device="cuda"), 4)
        db = torch.ones(N, device="cuda")
        J.jenga_linear_bwd(dy2, x2, w, act="relu", pre=pre, n_kept=torch.tensor([v], dtype=torch.int32, device="cuda"),
                           need=("dw", "db"), dw=dw, db=db, accumulate=True)
        X, W, D, Z = f64(x[:v]), f64(w), f64(dy[:v]), f64(pre[:v])
        _, rw, rb, dz = od.linear_bwd(D, X, W, "relu", Z)
        _, tw, tb = bwd_tols(X, W, D, dz, slope_err(Z, "relu"), v, "relu")
        close(dw, rw + 1, tw + 2 * U * (np.abs(rw) + 1))
        close(db, rb + 1, tb + 2 * U * (np.abs(rb) + 1))
    J.jenga_check_device_status()


def test_linear_fwd_extremes(J):
    # infinities and NaN stay in their row; saturated activations are exact
    x, w, b, _ = lin_case(40, 72, 64)
    clean, _ = J.jenga_linear_fwd(x, w, b, act="silu")
    x2 = x.clone()
    x2[3, 5], x2[9, 1] = NAN, float("inf")
    y, _ = J.jenga_linear_fwd(x2, w, b, act="silu")
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[[3, 9]] = False
    assert torch.equal(y[keep], clean[keep]) and torch.isnan(y[3]).all() and not torch.isfinite(y[9]).all()
    big = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    big[0, 0], big[1, 0] = 1000.0, -1000.0
    eye = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    eye[:, 0] = 1.0
    for kind in ("relu", "gelu", "silu"):
        y, _ = J.jenga_linear_fwd(big, eye, act=kind)
        assert (y[0] == 1000.0).all() and (y[1] == 0.0).all()
    J.jenga_check_device_status()


def bwd_tols(x, w, dy, dz, slope_err, rows, kind):
    """dz carries the slope's error; dx: bf16 dz against w over N terms; dw: exact or hi + lo dz
    (2^-16) over at most min(rows, 1024) truncated and rows / 1024 + 1 rounded adds; db: fp32."""
    X, W = np.abs(x), np.abs(w)
    D = np.abs(dz)
    e = np.abs(dy) * slope_err
    smooth = kind in ("gelu", "silu")
    N = w.shape[0]
    ex = (e + (RB * D if smooth else 0.0)) @ W + 2 * (N + 2) * U * (D @ W)
    n = min(2048 if smooth else 1024, rows) + rows / 512 + 4
    ew = (e + (2.0 ** -16 * D if smooth else 0.0)).T @ X + 2 * n * U * (D.T @ X)
    eb = e.sum(0) + (rows + 4) * U * D.sum(0)
    return ex * 1.01, ew * 1.01 + 1e-30, eb * 1.01 + 1e-30


def slope_err(z, kind):
    a = np.abs(z)
    if kind in ("none", "relu"):
        return np.zeros_like(z)
    return (24 + 3 * a + 2 * a * a) * U  # erff / __expf within a few + 1.173 z^2 / 2 ulp, slope <= 1.13


BWD_SIZES = [(1, 1, 1), (1, 64, 64), (3, 1541, 520), (65, 33, 72), (128, 128, 64), (257, 300, 1001), (300, 1541, 520),
             (600, 512, 256), (1100, 260, 136), (2500, 2304, 192), (4200, 64, 40)]


@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("M,N,K", BWD_SIZES)
def test_linear_bwd(J, M, N, K, kind):
    x, w, _, dy = lin_case(M, N, K)
    pre = randn(9, M, N, dt=torch.bfloat16, scale=1.5)
    pre[0, 0] = 0.0
    dx, dw, db = J.jenga_linear_bwd(dy, x, w, act=kind, pre=pre)
    J.jenga_check_device_status()
    X, W, D, Z = f64(x), f64(w), f64(dy), f64(pre)
    rx, rw, rb, dz = od.linear_bwd(D, X, W, kind, Z)
    tx, tw, tb = bwd_tols(X, W, D, dz, slope_err(Z, kind), M, kind)
    close(dx, rx, tx + RB * np.abs(rx) * 1.001 + 1e-30)
    close(dw, rw, tw)
    close(db, rb, tb)
    # the fp32 gradient is good to fp32-like accuracy as a whole, not only entry by entry
    if M > 1:
        assert np.linalg.norm(f64(dw) - rw) <= 1e-5 * np.linalg.norm(rw)
    # accumulate; any subset of outputs gives the same bits
    dw2, db2 = dw.clone(), db.clone()
    J.jenga_linear_bwd(dy, x, w, act=kind, pre=pre, need=("dw", "db"), dw=dw2, db=db2, accumulate=True)
    assert torch.equal(dw2, dw + dw) and torch.equal(db2, db + db)
    for need in (("dx",), ("dw",), ("db",), ("dx", "dw")):
        got = J.jenga_linear_bwd(dy, x, w, act=kind, pre=pre, need=need)
        for name, g, full in zip(("dx", "dw", "db"), got, (dx, dw, db)):
            assert (g is None) if name not in need else torch.equal(g, full)


@pytest.mark.parametrize("kind", ["none", "relu", "silu"])
def test_linear_bwd_device_count_and_pitches(J, kind):
    M, N, K, blk = 640, 300, 136, 16
    x, w, _, dy = lin_case(M, N, K)
    pre = randn(9, M, N, dt=torch.bfloat16)
    for n in (0, 1, 4, 23, 40):
        v = n * blk
        x2, dy2, pre2 = pitched(x, 8), pitched(dy, 3), pitched(pre, 5)
        for t in (x2, dy2, pre2):
            t[v:] = NAN
        nk = torch.tensor([n], dtype=torch.int32, device="cuda")
        dx = torch.full((M, K), 7.0, dtype=torch.bfloat16, device="cuda")
        dw = pitched(torch.zeros(N, K, device="cuda"), 3)
        _, _, db = J.jenga_linear_bwd(dy2, x2, w, act=kind, pre=pre2, n_kept=nk, blk=blk, dx=dx, dw=dw)
        J.jenga_check_device_status()
        assert (dx[v:] == 7.0).all() and torch.isnan(dw._base[:, K:]).all()
        if n == 0:
            assert not dw.any() and not db.any()
            continue
        X, W, D, Z = f64(x[:v]), f64(w), f64(dy[:v]), f64(pre[:v])
        rx, rw, rb, dz = od.linear_bwd(D, X, W, kind, Z)
        tx, tw, tb = bwd_tols(X, W, D, dz, slope_err(Z, kind), v, kind)
        close(dx[:v], rx, tx + RB * np.abs(rx) * 1.001 + 1e-30)
        close(dw, rw, tw)
        close(db, rb, tb)


def test_linear_bwd_segments_add_up(J):
    # the segment-wise use: gradients of consecutive row ranges accumulate into one fp32 buffer
    x, w, _, dy = lin_case(1000, 320, 200)
    pre = randn(9, 1000, 320, dt=torch.bfloat16)
    _, dw, db = J.jenga_linear_bwd(dy, x, w, act="relu", pre=pre)
    aw, ab = torch.zeros_like(dw), torch.zeros_like(db)
    for s in range(0, 1000, 384):
        e = min(s + 384, 1000)
        J.jenga_linear_bwd(dy[s:e], x[s:e], w, act="relu", pre=pre[s:e], need=("dw", "db"), dw=aw, db=ab, accumulate=True)
    X, W, D, Z = f64(x), f64(w), f64(dy), f64(pre)
    _, rw, rb, dz = od.linear_bwd(D, X, W, "relu", Z)
    _, tw, tb = bwd_tols(X, W, D, dz, slope_err(Z, "relu"), 1000, "relu")
    close(aw, rw, tw)
    close(ab, rb, tb)


# ------------------------------------------------------------------ dropout
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 8), (130, 256), (257, 1001), (33, 4096), (2000, 12)])
def test_dropout(J, rows, cols, dt):
    x, res = randn(cols, rows, cols, dt=dt), randn(cols + 1, rows, cols, dt=dt)
    for p, seed, off, r, row0 in ((0.1, 3, 5, None, 0), (0.5, 2 ** 63 + 11, 2 ** 40 + 3, res, 0),
                                  (0.25, -1, 2 ** 64 - 1, None, 2 ** 31 - rows), (0.0, 1, 1, res, 7), (1.0, 1, 1, res, 0),
                                  (1.0, 1, 1, None, 0)):
        y = J.jenga_dropout(x, p, seed, off, residual=r, row0=row0)
        J.jenga_check_device_status()
        m = (1 << 64) - 1
        want = od.dropout(f64(x), np.arange(rows, dtype=np.int64) + row0, p, seed & m, off & m,
                          f64(r) if r is not None else None)
        tol = HALF[dt] * np.abs(want) + 3 * U * (2 * np.abs(f64(x)) + np.abs(want) + np.abs(f64(res)))
        close(y, want, tol)
        if r is None:
            assert ((f64(y) != 0) == (want != 0)).all()


@pytest.mark.parametrize("h", [264, 265, 20])
def test_dropout_positions_segments_and_backward(J, h):
    S, blk, n = 1024, 64, 9
    x = randn(1, S, h, dt=torch.bfloat16)
    full = J.jenga_dropout(x, 0.3, 5, 6)
    idx, rows = kept(S, blk, n, 2)
    nk = torch.tensor([n - 2], dtype=torch.int32, device="cuda")
    out = torch.full((n * blk, h), 7.0, dtype=torch.bfloat16, device="cuda")
    y = J.jenga_dropout(x[rows].contiguous(), 0.3, 5, 6, idx=idx, n_kept=nk, blk=blk, out=out)
    v = (n - 2) * blk
    assert torch.equal(y[:v], full[rows][:v]) and (y[v:] == 7.0).all()  # a token's mask is its position's
    part = torch.cat([J.jenga_dropout(x[s:s + 300], 0.3, 5, 6, row0=s) for s in range(0, S, 300)])
    assert torch.equal(part, full)
    # dropped infinities and NaN leave no trace; in place on x and on the residual
    m = full == 0
    bad = torch.where(m, torch.full_like(x, NAN), x)
    bad[m & (torch.arange(h, device="cuda") % 2 == 0)] = float("inf")
    assert torch.equal(J.jenga_dropout(bad, 0.3, 5, 6), full)
    z = x.clone()
    J.jenga_dropout(z, 0.3, 5, 6, out=z)
    assert torch.equal(z, full)
    r = randn(3, S, h, dt=torch.bfloat16)
    want = J.jenga_dropout(x, 0.3, 5, 6, residual=r)
    J.jenga_dropout(x, 0.3, 5, 6, residual=r, out=r)
    assert torch.equal(r, want)
    # the backward is the same mask and scale on the gradient
    g = torch.ones_like(x)
    assert torch.equal(J.jenga_dropout(g, 0.3, 5, 6) != 0, full != 0)
    pit = pitched(x, 3)
    assert torch.equal(J.jenga_dropout(pit, 0.3, 5, 6), full)


# ------------------------------------------------------------------ large matrices
def test_offsets_beyond_32_bits(J):
    # every matrix below holds more than 2^31 elements: the last rows against the same rows alone
    bf = torch.bfloat16
    if torch.cuda.get_device_properties(0).total_memory < 60 << 30:
        pytest.skip("needs 40 GB of device memory")
    h, rows = 8192, (1 << 18) + 700
    x = torch.randn(1024, h, device="cuda").to(bf).repeat(rows // 1024 + 1, 1)[:rows]
    ga = randn(1, h, dt=bf)
    t = rows - 333
    y, mean, rstd = J.jenga_layernorm_fwd(x, ga)
    want = J.jenga_layernorm_fwd(x[t:].clone(), ga)
    assert torch.equal(y[t:], want[0]) and torch.equal(mean[t:], want[1])
    dx = J.jenga_layernorm_bwd(y, x, mean, rstd, ga, weight_grads=False)[0]
    assert torch.equal(dx[t:], J.jenga_layernorm_bwd(y[t:].clone(), x[t:].clone(), mean[t:].clone(), rstd[t:].clone(), ga,
                                                     weight_grads=False)[0])
    del dx
    J.jenga_dropout(x, 0.3, 5, 6, out=y)
    assert torch.equal(y[t:], J.jenga_dropout(x[t:].clone(), 0.3, 5, 6, row0=t))
    del x, y
    M, N, K = 200100, 11008, 64
    x, w = randn(2, M, K, dt=bf), randn(3, N, K, dt=bf, scale=0.2)
    y, pre = J.jenga_linear_fwd(x, w, act="relu", save_pre=True)
    v = M - 300
    ry, rz = od.linear_fwd(f64(x[v:]), f64(w), None, "relu")
    S = np.abs(f64(x[v:])) @ np.abs(f64(w)).T
    close(y[v:], ry, 2 * (K + 2) * U * S + RB * np.abs(ry) * 1.001 + 1e-30)
    close(pre[v:], rz, 2 * (K + 2) * U * S + RB * np.abs(rz) * 1.001 + 1e-30)
    dx, _, _ = J.jenga_linear_bwd(y, x, w, act="relu", pre=pre, need=("dx",))
    dy, z = f64(y[v:]), f64(pre[v:])
    rx = (dy * (z > 0)) @ f64(w)
    close(dx[v:], rx, 2 * (N + 2) * U * (np.abs(dy) @ np.abs(f64(w))) + RB * np.abs(rx) * 1.001 + 1e-30)
    J.jenga_check_device_status()


def test_dropout_more_rows_than_one_grid(J):
    rows, cols = 4 * 65535 + 300, 2048  # the grid holds 65535 steps of four rows of this width
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    y = J.jenga_dropout(x, 0.25, 9, 3)
    for s in (0, 4 * 65535 - 100, rows - 200):
        assert torch.equal(y[s:s + 200], J.jenga_dropout(x[s:s + 200], 0.25, 9, 3, row0=s))
    assert abs(float((y != 0).float().mean()) - 0.75) < 1e-3


# ------------------------------------------------------------------ streams, graphs, repeated calls
def _all_ops(J, t):
    y, mean, rstd = J.jenga_layernorm_fwd(t["x"], t["ga"], t["be"])
    a, pre = J.jenga_linear_fwd(y, t["w"], t["b"], act="gelu", save_pre=True)
    z = J.jenga_dropout(a, 0.2, 3, 4)
    dx, dw, db = J.jenga_linear_bwd(z, y, t["w"], act="gelu", pre=pre)
    return (y, mean, rstd, a, pre, z, dx, dw, db) + J.jenga_layernorm_bwd(dx, t["x"], mean, rstd, t["ga"])


def _inputs(seed):
    bf = torch.bfloat16
    return dict(x=randn(seed, 200, 264, dt=bf), ga=randn(1, 264, dt=bf), be=randn(2, 264, dt=bf),
                w=randn(3, 136, 264, dt=bf, scale=0.1), b=randn(4, 136))


def test_same_bits_on_repeats_side_stream_and_graph_replay(J):
    t, t2 = _inputs(0), _inputs(50)
    want, want2 = _all_ops(J, t), _all_ops(J, t2)
    for a, b in zip(_all_ops(J, t), want):
        assert torch.equal(a, b)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        side = _all_ops(J, t)
    s.synchronize()
    y = J.jenga_layernorm_fwd(t["x"], t["ga"], t["be"], stream=s)[0]  # the stream as an argument
    s.synchronize()
    assert torch.equal(y, want[0])
    for a, b in zip(side, want):
        assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = _all_ops(J, t)
    for k in t:
        t[k].copy_(t2[k])
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, want2):
        assert torch.equal(a, b)
    J.jenga_check_device_status()


def test_binding_refuses_what_the_kernels_cannot_read(J):
    bf = torch.bfloat16
    x, w = randn(0, 8, 64, dt=bf), randn(1, 16, 64, dt=bf)
    E = (ValueError, TypeError, J._lib.JengaError)
    for call in (lambda: J.jenga_linear_fwd(x.float(), w), lambda: J.jenga_linear_fwd(x, w[:, :32]),
                 lambda: J.jenga_linear_fwd(x.T, w), lambda: J.jenga_linear_fwd(x[:, 1:33], w[:, 1:33]),
                 lambda: J.jenga_linear_fwd(x, w, randn(2, 15)), lambda: J.jenga_linear_fwd(x, w, act="tanh"),
                 lambda: J.jenga_linear_fwd(x, w, out=torch.zeros(7, 16, dtype=bf, device="cuda")),
                 lambda: J.jenga_linear_fwd(x, w, residual=torch.zeros(8, 16, device="cuda")),
                 lambda: J.jenga_linear_bwd(x[:, :16], x, w, act="relu"),
                 lambda: J.jenga_linear_bwd(x[:, :16], x, w, accumulate=True),
                 lambda: J.jenga_linear_fwd(x, w, n_kept=torch.tensor([1], device="cuda"), blk=8),
                 lambda: J.jenga_layernorm_fwd(x.half()), lambda: J.jenga_layernorm_fwd(x, randn(2, 63)),
                 lambda: J.jenga_layernorm_fwd(x, randn(2, 64), randn(2, 64, dt=bf)),
                 lambda: J.jenga_layernorm_fwd(x, idx=torch.tensor([0], dtype=torch.int32, device="cuda"), blk=8,
                                               n_kept_max=2),
                 lambda: J.jenga_layernorm_fwd(x[:1].expand(8, 64)),
                 lambda: J.jenga_dropout(x, 1.5, 0), lambda: J.jenga_dropout(x, 0.5, 0, residual=x[:4]),
                 lambda: J.jenga_dropout(x, 0.5, 0, out=x.float()),
                 lambda: J.jenga_dropout(x, 0.5, 0, idx=torch.tensor([0], dtype=torch.int32, device="cuda"), blk=4)):
        with pytest.raises(E + (KeyError,)):
            call()
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert J.jenga_layernorm_fwd(x, idx=none, blk=8)[0].shape == (0, 64)
    empty = J.jenga_linear_fwd(x[:0], w)[0]
    assert empty.shape == (0, 16)
    _, dw, db = J.jenga_linear_bwd(empty, x[:0], w)
    assert not dw.any() and not db.any()
    assert J.jenga_dropout(x[:0], 0.5, 0).shape == (0, 64) and J.jenga_layernorm_fwd(x[:0])[0].shape == (0, 64)
    J.jenga_check_device_status()


# ------------------------------------------------------------------ a run of them, as used
def test_opt_style_sub_block_on_retained_rows(J):
    """x += dropout(relu(LN(x) w1^T + b1) w2^T + b2) on the kept blocks of a sequence, with the
    MLP criterion on the ReLU output, and every gradient, against float64 autograd."""
    bf = torch.bfloat16
    S, blk, h, F, nb = 512, 32, 256, 520, 16
    X = randn(0, S, h, dt=bf)
    ga, be = randn(1, h, dt=bf, scale=0.2, shift=1.0), randn(2, h, dt=bf, scale=0.2)
    w1, b1 = randn(3, F, h, dt=bf, scale=0.1), randn(4, F, dt=bf, scale=0.2)
    w2, b2 = randn(5, h, F, dt=bf, scale=0.1), randn(6, h, dt=bf, scale=0.2)
    idx, nk, _ = J.jenga_select(randn(7, nb), "topk", 9)
    n = 9
    G = randn(8, S, h, dt=bf)

    y, mean, rstd = J.jenga_layernorm_fwd(X, ga, be, idx=idx, n_kept=nk, blk=blk, n_kept_max=n)
    a, _ = J.jenga_linear_fwd(y, w1, b1, act="relu", n_kept=nk, blk=blk)
    crit = J.jenga_mlp_block_scores(a, blk, nk)
    o, _ = J.jenga_linear_fwd(a, w2, b2, n_kept=nk, blk=blk)
    d = J.jenga_dropout(o, 0.1, 11, 12, idx=idx, n_kept=nk, blk=blk)
    out = X.clone()
    J.jenga_scatter_add(out, d, idx, nk, blk)

    Gk = J.jenga_gather(G, idx, nk, blk, n * blk)
    do = J.jenga_dropout(Gk, 0.1, 11, 12, idx=idx, n_kept=nk, blk=blk)
    da, dw2, db2 = J.jenga_linear_bwd(do, a, w2, n_kept=nk, blk=blk)
    dn, dw1, db1 = J.jenga_linear_bwd(da, y, w1, act="relu", pre=a, n_kept=nk, blk=blk)
    dX = G.clone()
    _, dga, dbe = J.jenga_layernorm_bwd(dn, X, mean, rstd, ga, idx=idx, n_kept=nk, blk=blk, n_kept_max=n, dres=dX, dx=dX)
    J.jenga_check_device_status()

    rows = (idx[:n].long().cpu()[:, None] * blk + torch.arange(blk)[None]).reshape(-1)
    t = {k: v.double().cpu().requires_grad_() for k, v in dict(X=X, ga=ga, be=be, w1=w1, b1=b1, w2=w2, b2=b2).items()}
    ln = torch.nn.functional.layer_norm(t["X"][rows], (h,), t["ga"], t["be"])
    act = torch.relu(ln @ t["w1"].T + t["b1"])
    keep = torch.from_numpy(od.dropout_mask(rows.numpy(), h, 0.1, 11, 12)).double()
    scale = 65536.0 / (65536 - od.dropout_threshold(0.1))
    ref = t["X"].index_add(0, rows, (act @ t["w2"].T + t["b2"]) * keep * scale)
    ref.backward(G.double().cpu())

    def rel(got, want):
        return float(np.linalg.norm(f64(got) - want.detach().numpy()) / np.linalg.norm(want.detach().numpy()))

    # Norm-wise bars.  out and dX end in one bf16 rounding (2^-8).  Inside, ln, a, o and d (then
    # do, da, dn) are bf16 tensors: at most four more roundings, each at most 2^-8 of the
    # tensor it rounds; a ReLU whose pre-activation changes sign under them passes or drops a
    # value no larger than that error.  So 5 roundings bound everything with a factor two for
    # the products' own amplification of errors that are not aligned with their output.
    bar = 2 * 5 * RB
    assert rel(crit, act.reshape(n, -1).abs().sum(1)) < bar
    for got, want in ((out, ref), (dX, t["X"].grad), (dga, t["ga"].grad), (dbe, t["be"].grad), (dw1, t["w1"].grad),
                      (db1, t["b1"].grad), (dw2, t["w2"].grad), (db2, t["b2"].grad)):
        assert rel(got, want) < bar
    other = torch.ones(S, dtype=torch.bool)
    other[rows] = False
    assert torch.equal(out[other.cuda()], X[other.cuda()]) and torch.equal(dX[other.cuda()], G[other.cuda()])
