"""What the vocabulary losses' workspaces come to, without a GPU."""
import pytest


@pytest.fixture(scope="module")
def pg():
    from hashed_head_gram_gb300.build import build
    build()
    from hashed_head_gram_gb300 import pg as mod
    return mod


# What a call keeps beside its chunk of rows: 24 bytes a row for references, sums and factors and 16 a tile of 256 columns (a
# chunk of narrow rows has many), and parts of the gradients (640 tiles of 256 x 256 in fp32 of each)
def beside(N, V, d):
    rows = min(N, (2 << 30) // (2 * V) + 256)
    return rows * (24 + 16 * ((V + 255) // 256)) + 2 * 640 * 4 * 256 * 256 + 4 * V * d + (1 << 20)


@pytest.mark.parametrize("K", [1, 30, 256])
@pytest.mark.parametrize("V,d", [(64, 96), (300, 8), (1000, 96), (50304, 768), (128000, 33)])
def test_lists_count_among_what_is_kept_of_a_chunk(pg, V, d, K):
    for N in (4096, 1 << 20, 1 << 22, (1 << 31) - 1):
        for hd, wd, ghd, gwd in [(1, 1, 1, 1), (1, 1, None, 0), (0, 1, 0, None)]:
            size = pg.vocab_distill_grad_workspace_size(N, V, d, K, hd, wd, ghd, gwd)
            copies = 2 * 3 * V * (d + 64)  # of an odd table, and a chunk's sum of its gradient
            assert size <= (2 << 30) + beside(N, V, d) + copies, (N, size)


def test_forward_lists_are_bounded(pg):
    for N in (1 << 20, (1 << 31) - 1):
        assert pg.vocab_distill_workspace_size(N, 64, 96, 256, 1, 1) <= 1 << 28
        assert pg.vocab_distill_workspace_size(N, 50304, 768, 256, 1, 1) <= 1 << 28


def test_few_rows_reserve_their_own(pg):
    # U and the sums of the rows that there are (to eight), not of a tile of 256
    V = (1 << 24) - 1
    assert pg.vocab_ce_grad_workspace_size(1, V, 8, 1, 1, None, 0) <= 8 * (6 * V + V // 4 + 64) + (1 << 20)
    assert pg.vocab_ce_grad_workspace_size(8, 128000, 2560, 1, 1, 1, 1) <= 8 * (2 * 128000 + 128000 // 4) + 4 * 8 * 2560 * 64 + (1 << 20)
    assert pg.vocab_distill_grad_workspace_size(1, 1000, 64, 256, 1, 1, 1, 0) <= 1 << 19
    for N, V, d in [(1, 5000, 64), (31, 50304, 768), (128, 50304, 768)]:
        few = -(-N // 8) * 8
        for hd, wd, ghd, gwd in [(1, 1, 1, 1), (0, 0, 0, 0)]:
            size = pg.vocab_ce_grad_workspace_size(N, V, d, hd, wd, ghd, gwd)
            parts = 4 * few * d * max(32, 304 // -(-d // 128) + 1)
            assert size <= few * (6 * (V + 64) + V // 2 + 24 * d) + parts + 6 * V * d + (1 << 20), (N, size)
