"""Scoring repeats bit for bit.  Its query and key tiles pass through rings whose stages two issuing
warps use in turn; q and k larger than L2, read again from memory in every call, vary the order in which
copies land."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def J():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import token_sparse_long_b200 as J
    J._lib.load()
    return J


@pytest.mark.parametrize("mode,S,heads,blk", [("paper_blockmax", 8192, 32, 64), ("paper_blockmax", 1000 * 32, 5, 32),
                                              ("softmax_mass", 8192, 32, 64), ("softmax_mass", 4096 + 32, 33, 32)])
def test_scores_repeat_bit_for_bit(J, mode, S, heads, blk):
    g = torch.Generator(device="cuda").manual_seed(S + heads)
    qk = (torch.randn(S, 2 * heads * 128, generator=g, device="cuda")).to(torch.bfloat16)
    q, k = qk[:, :heads * 128], qk[:, heads * 128:]
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    first = None
    for i in range(12):
        flush.fill_(i)
        sc = J.jenga_score_blocks(q, k, heads, 128, blk, mode=mode).clone()
        first = sc if first is None else first
        assert torch.equal(sc, first), i
    J.jenga_check_device_status()
    assert torch.isfinite(first).all()
