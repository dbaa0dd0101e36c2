"""The vocabulary losses where their rows come in chunks and their gradients in parts."""
import pytest
import torch

from tests.test_gpu_vocab import BF16, F32, check_grads, check_values, make, reference, run_distill

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,V,d,K,ghd,gwd", [(6000, 70001, 40, 30, F32, BF16), (700_000, 64, 40, 256, BF16, BF16), (700_000, 64, 33, 200, None, F32)])
def test_lists_in_chunks(cuda, N, V, d, K, ghd, gwd):
    # 2 GiB hold 4800 rows of three pieces of 70,001 columns, or some 640,000 of 64 with lists of 256
    gen = torch.Generator(device=cuda).manual_seed(N + K)
    h, W, _ = make(3, 1, V, d, BF16, BF16, cuda)
    h = torch.randn(N, d, generator=gen, device=cuda).to(BF16)
    ids = torch.randint(-V // 8, V, (N, K), generator=gen, device=cuda, dtype=torch.int32)
    u = (torch.randn(N, K, generator=gen, device=cuda) * 2).to(BF16)
    r = reference(h, W, ids=ids, u=u, grad_scale=0.01)
    loss, lse, dh, dW = run_distill(h, W, ids, u, ghd, gwd, grad_scale=0.01)
    check_values(r, loss, lse)
    check_grads(r, dh, dW)
