"""Sizes at the limits of the products around the finalize, where row numbers and
steps of k come near 2^31."""
import pytest
import torch

import ffn_ref as R

BF16 = torch.bfloat16
MOST = 2 ** 31 - 1


@pytest.mark.gpu
def test_row_map_that_ends_at_the_last_row(cuda_lib):
    """One token, tiles of 2^31 - 1 rows: the experts behind its own begin, and
    end, at the last row, and have no padding to write."""
    for E, expert in ((2, 0), (2, 1), (40, 0)):
        ids = torch.tensor([[expert]], dtype=torch.int32, device="cuda")
        m = cuda_lib.permute_tokens(ids, E, MOST)
        assert m["idx_map"].tolist() == [[0]]
        assert m["offsets"].tolist() == [0] * (expert + 1) + [MOST] * (E - expert)
        assert m["counts"].tolist() == [int(e == expert) for e in range(E)]
        token = m["row_token"]
        assert token.numel() == MOST and int(token[0]) == 0
        for at in range(1, MOST, 2 ** 28):      # in pieces: comparisons are 64-bit indexed
            assert bool((token[at:at + 2 ** 28] == -1).all())
        del m, token


@pytest.mark.gpu
def test_weight_gradient_over_the_most_rows(cuda_lib):
    """2^31 - 1 rows, which dweight sums over: a few carry values, the first and
    last blocks of 64 among them, the others are zeros and add nothing."""
    N, K = 8, 8
    x = torch.zeros(MOST, K, dtype=BF16, device="cuda")
    dout = torch.zeros(MOST, N, dtype=BF16, device="cuda")
    some = [0, 1, 63, 64, 2 ** 30, MOST - 64, MOST - 63, MOST - 33, MOST - 32, MOST - 2, MOST - 1]
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    for t in (x, dout):
        t[some] = torch.randn(len(some), 8, device="cuda", generator=g).to(BF16)
    w = torch.ones(N, K, dtype=BF16, device="cuda")
    got = cuda_lib.linear_backward(dout, x, w, want_dx=False, want_dbias=True)
    R.check(got, R.backward(dout[some], x[some], w, None, "none", False))
    assert cuda_lib.lost_waits() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("N", [8, 24])
def test_products_over_the_most_rows(cuda_lib, N):
    """2^31 - 1 rows forward and through dx: nothing in the tiles' places may pass 31
    bits.  A few rows carry values, the first and last tiles' among them."""
    K = 8
    x = torch.zeros(MOST, K, dtype=BF16, device="cuda")
    some = [0, 1, 255, 256, 2 ** 30, MOST - 257, MOST - 256, MOST - 33, MOST - 2, MOST - 1]
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x[some] = torch.randn(len(some), K, device="cuda", generator=g).to(BF16)
    w = torch.randn(N, K, device="cuda", generator=g).to(BF16)

    def zeros_elsewhere(out):
        assert int(out[:2 ** 20].count_nonzero(dim=1).bool().sum()) == 4
        assert int(out[-2 ** 20:].count_nonzero(dim=1).bool().sum()) == 5
        assert int(out[2 ** 30 - 1000:2 ** 30 + 1000].count_nonzero(dim=1).bool().sum()) == 1

    out = cuda_lib.linear(x, w)["out"]
    R.check({"out": out[some]}, {"out": R.linear(x[some], w)["out"]})
    zeros_elsewhere(out)
    if N == K:
        dx = cuda_lib.linear_backward(x, x, w, want_dweight=False, dx=out)["dx"]
        R.check({"dx": dx[some]}, {"dx": R.backward(x[some], x[some], w, None, "none", False)["dx"]})
        zeros_elsewhere(dx)
    assert cuda_lib.lost_waits() == 0
