"""Sizes at the limits of the products around the finalize, where row numbers and
steps of k come near 2^31."""
import pytest
import torch

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
