"""Layer norm, linear layer and dropout where their kernels' rings wrap, their row counts, values
and sizes end: against the same formulas in float64.

U = 2^-24 is half an fp32 step and RB = 2^-8 half a bf16 step, relative to the value; a sum of n
fp32 terms is off by at most n U times the sum of magnitudes, on the tensor core, which
truncates, by 2 n U."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U, RB = 2.0 ** -24, 2.0 ** -8
BF = torch.bfloat16


@pytest.fixture(scope="module")
def J():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import token_sparse_long_b200 as J
    J._lib.load()
    return J


def randn(seed, *shape, dt=BF, scale=1.0, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale + shift).to(dt)


def close(got, want, tol):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), float((err / tol).nan_to_num().max()), bad.nonzero()[:4].tolist())


# ------------------------------------------------------------------ rings that wrap
@pytest.mark.parametrize("M", [1, 2])
@pytest.mark.parametrize("N,K", [(11008, 2560), (11003, 3584), (11008, 5120), (9001, 7168), (11008, 13824), (5000, 16384),
                                 (40000, 72)])
def test_linear_rows_ring_wraps(J, M, N, K):
    """One or two rows of x: every SM takes several times as many rows of w as its ring holds."""
    x, w, b = randn(1, M, K), randn(2, N, K, scale=1.5 / K ** 0.5), randn(3, N, dt=torch.float32)
    y, pre = J.jenga_linear_fwd(x, w, b, save_pre=True)
    J.jenga_check_device_status()
    want = x.double() @ w.double().T + b.double()
    S = x.double().abs() @ w.double().abs().T + b.double().abs()
    # fp32 sums of at most K / 64 + 40 sequential adds a lane
    close(y, want, (K / 64 + 40) * U * S + RB * want.abs() * 1.001)
    assert torch.equal(y, pre)
    for _ in range(3):
        assert torch.equal(J.jenga_linear_fwd(x, w, b)[0], y)


@pytest.mark.parametrize("M,N,K", [(16, 32000, 2880), (50, 40000, 320), (100, 40000, 960), (20000, 128, 320), (16, 40000, 40),
                                   (128, 40001, 64), (20000, 100, 64), (9, 33000, 200)])
def test_linear_odd_k_blocks_and_several_tiles_a_cluster(J, M, N, K):
    """Products whose tiles have an odd number of 64-deep k-blocks and of which a CTA pair takes
    several: the two issuing warps change places from tile to tile."""
    x, w, b = randn(1, M, K), randn(2, N, K, scale=1.5 / K ** 0.5), randn(3, N, dt=torch.float32)
    y, _ = J.jenga_linear_fwd(x, w, b)
    J.jenga_check_device_status()
    want = x.double() @ w.double().T + b.double()
    S = x.double().abs() @ w.double().abs().T + b.double().abs()
    close(y, want, 2 * (K + 4) * U * S + RB * want.abs() * 1.001)
    for _ in range(3):
        assert torch.equal(J.jenga_linear_fwd(x, w, b)[0], y)


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("M,N,K", [(832, 1024, 4096), (40, 1024, 4096), (200, 1100, 3904), (16, 2880, 32000), (100, 960, 20000)])
def test_linear_bwd_odd_k_blocks_and_several_tiles_a_cluster(J, M, N, K, act):
    x, w, dy, z = randn(1, M, K), randn(2, N, K, scale=1.5 / N ** 0.5), randn(3, M, N), randn(4, M, N)
    dx, dw, db = J.jenga_linear_bwd(dy, x, w, act=act, pre=None if act == "none" else z)
    J.jenga_check_device_status()
    dz, e = dy.double(), 0.0
    if act == "silu":
        s = torch.sigmoid(z.double())
        dz = dz * s * (1 + z.double() * (1 - s))
        # __expf is within 2 + 1.173 |z| ulp; slope <= 1.13, the products round a few times
        e = dy.double().abs() * (24 + 3 * z.double().abs()) * U
    D, X, W = dz.abs(), x.double().abs(), w.double().abs()
    smooth = RB if act == "silu" else 0.0  # dx takes dz as one bf16 operand
    want = dz @ w.double()
    close(dx, want, 1.01 * ((e + smooth * D) @ W + 2 * (N + 4) * U * (D @ W)) + RB * want.abs() * 1.001 + 1e-30)
    n = min(512, M) + M / 512 + 8
    close(dw, dz.T @ x.double(), 1.01 * ((e + 2 * U * D).T @ X + 2 * n * U * (D.T @ X)) + 1e-30)
    close(db, dz.sum(0), ((e + D * 0).sum(0) + (M + 4) * U * D.sum(0)) * 1.01)
    for _ in range(3):
        for a, b in zip(J.jenga_linear_bwd(dy, x, w, act=act, pre=None if act == "none" else z), (dx, dw, db)):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ counts near 2^31
def test_layernorm_as_many_rows_as_an_int_holds(J):
    if torch.cuda.get_device_properties(0).total_memory < 60 << 30:
        pytest.skip("needs 40 GB of device memory")
    rows = 2 ** 31 - 1
    x = torch.ones(rows, 1, dtype=BF, device="cuda")
    dy = torch.zeros(rows, 1, dtype=BF, device="cuda")
    at = torch.tensor([0, 1, 2 ** 30, rows - 2400, rows - 2, rows - 1], device="cuda")
    dy[at] = 1.0
    mean, rstd = (torch.full((rows,), v, device="cuda") for v in (0.5, 2.0))
    # h = 1, n = (1 - 1/2) 2 = 1: dx = rstd (g - g - n g n) = -2 dy, exact in every step
    dx, dg, db = J.jenga_layernorm_bwd(dy, x, mean, rstd)
    J.jenga_check_device_status()
    assert (dx[at] == -2.0).all() and float(dg) == 6.0 and float(db) == 6.0
    assert int((dx != 0).sum()) == 6
    del dx, dy, mean, rstd
    y, mean, rstd = J.jenga_layernorm_fwd(x, eps=0.25)
    J.jenga_check_device_status()
    assert not y.any() and bool((mean == 1.0).all()) and bool((rstd == 2.0).all())


# ------------------------------------------------------------------ infinities, NaN, far tails
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("M,N,K", [(200, 72, 64), (200, 67, 64)])
def test_linear_bwd_infinite_and_nan_gradients(J, act, M, N, K):
    """An infinite dz makes its row of dw infinite, its column of db and its row of dx; a NaN makes them NaN."""
    x, w, dy = randn(1, M, K), randn(2, N, K), randn(3, M, N)
    z = randn(4, M, N).abs() + 0.5  # slopes above 0
    dy[7, 3], dy[9, 5], dy[30, 40] = math.inf, -math.inf, math.nan
    dx, dw, db = J.jenga_linear_bwd(dy, x, w, act=act, pre=None if act == "none" else z)
    J.jenga_check_device_status()
    assert torch.equal(dw[3], x[7].float() * math.inf) and torch.equal(dw[5], x[9].float() * -math.inf)
    assert db[3] == math.inf and db[5] == -math.inf
    assert torch.isnan(dw[40]).all() and torch.isnan(db[40]) and torch.isnan(dx[30]).all()
    assert torch.equal(dx[7].float(), w[3].float() * math.inf) and torch.equal(dx[9].float(), w[5].float() * -math.inf)
    rest = torch.ones(N, dtype=torch.bool, device="cuda")
    rest[[3, 5, 40]] = False
    assert torch.isfinite(dw[rest]).all() and torch.isfinite(db[rest]).all()
    rows = torch.ones(M, dtype=torch.bool, device="cuda")
    rows[[7, 9, 30]] = False
    assert torch.isfinite(dx[rows]).all()


def _phi(z):  # (ndtr cancels in the lower tail)
    return 0.5 * torch.special.erfc(z * -math.sqrt(0.5)), torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)


@pytest.mark.parametrize("M", [1, 3, 300])
@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_activation_tails_are_relatively_exact(J, act, M):
    """y = act(z) for one z a column, far into the tail where act(z) is tiny: a bf16 rounding and a
    few fp32 ones relative to y itself.  erfcf is within 4 ulp, its rounded argument adds
    1.3 (1 + z^2) half ulp; __expf is within 2 + 1.173 |z| ulp."""
    lo = -12.0 if act == "gelu" else -80.0
    z = torch.linspace(lo, 8.0, 520, device="cuda").to(BF)
    w = torch.zeros(520, 8, dtype=BF, device="cuda")
    w[:, 0] = z
    x = torch.zeros(M, 8, dtype=BF, device="cuda")
    x[:, 0] = 1.0
    y, _ = J.jenga_linear_fwd(x, w, act=act)
    J.jenga_check_device_status()
    Z = z.double()
    want = Z * _phi(Z)[0] if act == "gelu" else Z * torch.sigmoid(Z)
    rel = (1.3 * (1 + Z * Z) + 16) * U if act == "gelu" else (10 + 2.4 * Z.abs()) * U
    close(y, want.expand(M, -1), (want.abs() * (rel + RB * 1.001)).expand(M, -1))
    assert (y[0][z < -4] != 0).all()


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_activation_slopes_in_the_tails_and_at_infinity(J, act):
    z = torch.linspace(-12.0, 8.0, 518, device="cuda").to(BF)
    z = torch.cat([z, torch.tensor([math.inf, -math.inf], device="cuda", dtype=BF)])[None].contiguous()
    dy = torch.ones_like(z)
    x, w = randn(1, 1, 8), randn(2, 520, 8)
    dx, dw, db = J.jenga_linear_bwd(dy, x, w, act=act, pre=z)
    J.jenga_check_device_status()
    assert db[518] == 1.0 and db[519] == 0.0
    assert torch.isfinite(dx).all() and torch.equal(dw[518], x[0].float()) and not dw[519].any()
    Z = z[0, :518].double()
    if act == "gelu":
        P, f = _phi(Z)
        want = P + Z * f
        tol = P * (1.3 * (1 + Z * Z) + 12) * U + (Z * f).abs() * (2.2 * Z * Z + 14) * U
    else:
        s = torch.sigmoid(Z)
        want = s * (1 + Z * (1 - s))
        # s carries the exponential's error; 1 - s and 1 + z (1 - s) add roundings of their operands
        tol = (s + (Z * s * (1 - s)).abs() + (Z * s * s).abs()) * (12 + 2.4 * Z.abs()) * U
    close(db[:518], want, tol)
    # three bf16 parts: two truncated adds and a rounded one on top of dz's error
    close(dw[:518], want[:, None] * x.double(), (tol + 8 * U * want.abs())[:, None] * x.double().abs() + 1e-30)


# ------------------------------------------------------------------ columns of one matrix
def test_inputs_and_outputs_side_by_side_in_one_matrix(J):
    M, K, N = 300, 264, 200
    b = torch.full((M, K + N + N + 8), math.nan, dtype=BF, device="cuda")
    x, y, pre = b[:, :K], b[:, K:K + N], b[:, K + N:K + 2 * N]
    w, dy = randn(2, N, K, scale=0.1), randn(3, M, N)
    x0 = randn(1, M, K)
    x.copy_(x0)
    want, wpre = J.jenga_linear_fwd(x0, w, act="gelu", save_pre=True)
    J.jenga_linear_fwd(x, w, act="gelu", out=y, pre=pre)
    assert torch.equal(y, want) and torch.equal(pre, wpre) and torch.equal(x, x0)
    ref = J.jenga_linear_bwd(dy, x0, w, act="gelu", pre=wpre)
    y.copy_(dy)
    dx = torch.full((M, 2 * K), math.nan, dtype=BF, device="cuda")
    dx[:, K:] = x0
    got = J.jenga_linear_bwd(y, dx[:, K:], w, act="gelu", pre=pre, dx=dx[:, :K])
    assert all(torch.equal(a, c) for a, c in zip(got, ref)) and torch.equal(dx[:, K:], x0)
    ln = torch.full((M, 2 * K), math.nan, dtype=BF, device="cuda")
    ln[:, :K] = x0
    J.jenga_layernorm_fwd(ln[:, :K], out=ln[:, K:])
    assert torch.equal(ln[:, K:], J.jenga_layernorm_fwd(x0)[0]) and torch.equal(ln[:, :K], x0)
    J.jenga_dropout(ln[:, :K], 0.3, 5, 6, out=ln[:, K:])
    assert torch.equal(ln[:, K:], J.jenga_dropout(x0, 0.3, 5, 6)) and torch.equal(ln[:, :K], x0)
    assert torch.isnan(b[:, K + 2 * N:]).all()
    J.jenga_check_device_status()


@pytest.mark.parametrize("M,N,K", [(1, 300, 521), (1, 700, 8191), (40, 1, 521), (1, 1, 3), (300, 1, 77)])
def test_linear_single_rows_of_any_length(J, M, N, K):
    """One row of x, or of w, as it lies: its stride is no multiple of eight elements."""
    P = (K + 7) // 8 * 8
    x = randn(1, 1, K) if M == 1 else randn(1, M, P)[:, :K]
    w = randn(2, 1, K, scale=0.1) if N == 1 else randn(2, N, P, scale=0.1)[:, :K]
    dy = randn(3, M, N)
    y, _ = J.jenga_linear_fwd(x, w)
    dx, dw, db = J.jenga_linear_bwd(dy, x, w)
    J.jenga_check_device_status()
    X, W, D = x.double(), w.double(), dy.double()
    close(y, X @ W.T, 2 * (K + 4) * U * (X.abs() @ W.abs().T) + RB * (X @ W.T).abs() * 1.001)
    close(dx, D @ W, 2 * (N + 4) * U * (D.abs() @ W.abs()) + RB * (D @ W).abs() * 1.001 + 1e-30)
    close(dw, D.T @ X, 2 * (M + 4) * U * (D.abs().T @ X.abs()) + 1e-30)
    close(db, D.sum(0), (M + 4) * U * D.abs().sum(0) + 1e-30)


@pytest.mark.parametrize("M", [1, 2, 16, 300])
def test_relu_keeps_nan_and_infinity(J, M):
    w = torch.zeros(72, 64, dtype=BF, device="cuda")
    w[:, 0] = 1.0
    x = torch.zeros(M, 64, dtype=BF, device="cuda")
    for v, want in ((math.nan, math.nan), (math.inf, math.inf), (-math.inf, 0.0), (-3.0, 0.0), (2.0, 2.0)):
        x[M - 1, 0] = v
        b = torch.zeros(72, device="cuda")
        y = J.jenga_linear_fwd(x, w, b, act="relu")[0][M - 1].float()
        z = torch.full((72,), v, device="cuda")
        assert torch.equal(torch.isnan(y), torch.isnan(z)), v
        if not math.isnan(v):
            assert (y == want).all(), v
    J.jenga_check_device_status()


# ------------------------------------------------------------------ dw as an fp32 result
@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("M,N,K", [(4096, 520, 264), (4096, 2304, 1024)])
def test_linear_dw_holds_all_bits_of_a_smooth_dz(J, act, M, N, K):
    """dw's error as a whole.  dz is within about 8 half steps of fp32 (its slope's evaluation) and held in
    24 bits; 512 products a time lose 5e-7 in the truncating accumulator: together below 1.1e-6.
    With dz in 16 bits it is 4e-6, and so it is with 4096 products in one accumulator."""
    x, dy, z = randn(1, M, K), randn(2, M, N), randn(3, M, N)
    dw = J.jenga_linear_bwd(dy, x, randn(4, N, K), act=act, pre=z, need=("dw",))[1]
    J.jenga_check_device_status()
    Z = z.double()
    if act == "gelu":
        P, f = _phi(Z)
        dz = dy.double() * (P + Z * f)
    else:
        s = torch.sigmoid(Z)
        dz = dy.double() * s * (1 + Z * (1 - s))
    want = dz.T @ x.double()
    assert float((dw.double() - want).norm() / want.norm()) < 1.5e-6


@pytest.mark.parametrize("N,K", [(512, 256), (2304, 2304)])
def test_linear_dw_of_many_positive_rows(J, N, K):
    """All products positive, so truncation adds up.  512 of them enter an accumulator in 32 steps of 16;
    a step truncates the aligned products and the sum, each by less than 2^-23 of the sum so far, half the
    chunk's on average: 2 * 32 * 2^-23 / 2 = 3.8e-6; the chunks' sums are added with rounding, 32 half
    steps of half the total: 1e-6.  db adds at most 8 + 8 + 256 sums in a row.  In one accumulator 16384 rows would lose about 5e-5."""
    M = 16384
    x, dy = randn(1, M, K).abs() + 0.25, randn(2, M, N).abs() + 0.25
    _, dw, db = J.jenga_linear_bwd(dy, x, randn(4, N, K), need=("dw", "db"))
    J.jenga_check_device_status()
    want = dy.double().T @ x.double()
    assert float(((dw.double() - want) / want).abs().max()) < 4.9e-6
    close(db, dy.double().sum(0), 280 * U * dy.double().sum(0))


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_linear_bwd_without_dw_in_the_smaller_workspace(J, act):
    M, N, K = 700, 328, 264
    x, w, dy, z = randn(1, M, K), randn(2, N, K, scale=0.1), randn(3, M, N), randn(4, M, N)
    full = J.jenga_linear_bwd(dy, x, w, act=act, pre=z)
    n = J._lib.load().jenga_linear_bwd_workspace_bytes(M, N, K, J._lib.ACT_RELU)
    buf = torch.full((n + 4096,), 170, dtype=torch.uint8, device="cuda")
    dx, dw, db = J.jenga_linear_bwd(dy, x, w, act=act, pre=z, need=("dx", "db"), ws=buf[:n])
    assert dw is None and torch.equal(dx, full[0]) and torch.equal(db, full[2])
    assert (buf[n:] == 170).all()
    J.jenga_check_device_status()
