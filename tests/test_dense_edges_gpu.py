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
