"""The teacher's softmax at both ends of its type: what counts are a list's differences, not its sizes."""
import math

import pytest
import torch

from tests.test_gpu_vocab import BF16, F32, check_grads, check_values, make, reference, run_distill

pytestmark = pytest.mark.gpu


def differences(u, T):
    """What each logit of a list is below its largest, in 64 bits. Below 100 T a weight is e^-100 at most, nothing beside
    the 2^-126 of check_grads: those are held there, so that the reference's tolerance is that of the tokens with weight."""
    u = u.double()
    top = u.amax(1, keepdim=True)
    return torch.where(u == -math.inf, u, (u - torch.where(top == -math.inf, 0.0, top)).clamp(min=-100 * T))


def lists(N, K, udt, cuda, T):
    """Lists at the ends of the type: (name, logits), a row each, over and over."""
    low, high = torch.finfo(udt).min, torch.finfo(udt).max
    gen = torch.Generator().manual_seed(N + K)
    u = torch.empty(N, K)
    for i in range(N):
        row = torch.randn(K, generator=gen) * 2
        kind = i % 8
        if kind == 0:
            row[:] = low                     # even weights
        elif kind == 1:
            row[:] = high
        elif kind == 2:
            row[:] = low
            row[0] = row[K // 2] = high      # two even weights
        elif kind == 3:
            row[1:] = low                    # a weight of one
        elif kind == 4:
            row[:] = low
            row[::2] = -math.inf             # even weights of the others
        elif kind == 5:
            row[:] = 0.9 * low               # (0.9 low is another value of the type: a weight of one)
            row[K - 1] = 0.5 * low
        elif kind == 6:
            row += 3e4                       # differences that the size hides from a quotient
        u[i] = row
    return u.to(udt).to(cuda)


@pytest.mark.parametrize("udt", [F32, BF16])
@pytest.mark.parametrize("T", [0.3, 0.7, 1.0, 3.0])
@pytest.mark.parametrize("N,V,K", [(5, 700, 40), (100, 700, 7), (300, 700, 130)])
def test_lists_at_the_ends_of_their_type(cuda, N, V, K, T, udt):
    h, W, _, ids, _ = make(N + K, N, V, 80, BF16, BF16, cuda, K=K, pad=0.0)
    ids[ids < 0] = 3
    u = lists(N, K, udt, cuda, T)
    r = reference(h, W, ids=ids, u=differences(u, T), T=T, grad_scale=0.5)
    assert r["keep"].all() and float(r["E"].max()) < 2e-3  # (a tolerance of ordinary size)
    loss, lse, _, _ = run_distill(h, W, ids, u, temperature=T)
    check_values(r, loss, lse)
    for gwd in (BF16, F32):
        loss, lse, dh, dW = run_distill(h, W, ids, u, BF16, gwd, temperature=T, grad_scale=0.5)
        check_values(r, loss, lse)
        check_grads(r, dh, dW)


def test_differences_past_the_type(cuda):
    # u - max u passes fp32's range, (u - max u) / T does not
    N, V, K, T = 40, 700, 6, 2.5e38
    h, W, _, ids, _ = make(7, N, V, 80, BF16, BF16, cuda, K=K, pad=0.0)
    ids[ids < 0] = 3
    u = torch.linspace(-3.2e38, 3.2e38, K, dtype=torch.float64).float().to(cuda).repeat(N, 1)
    r = reference(h, W, ids=ids, u=differences(u, T), scale=T, T=T, grad_scale=0.5)
    loss, lse, dh, dW = run_distill(h, W, ids, u, BF16, F32, scale=T, temperature=T, grad_scale=0.5)
    check_values(r, loss, lse)
    check_grads(r, dh, dW)
