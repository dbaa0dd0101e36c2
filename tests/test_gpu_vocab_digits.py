"""Digits that the vocabulary losses keep where a row's logits, or its weight, are far from one.

Tolerances. p = exp(z - lse) and 1 - p, the sum of the other tokens' exponentials over all, are sums and quotients of
exponentials of differences. An exponential has a relative error of 2^-22 from its own function, one of its argument's rounding
(2^-23 of the difference, twice: scale log2(e) has one too) and the sum of V terms 300 roundings; so a relative
REL = 2^-22 (2 difference + 80) of each of dz's parts, and of a loss as far as it comes of exponentials. On top comes twice what the
logits themselves are off, which is nothing where all their products and sums are whole numbers."""
import math

import pytest
import torch

from tests.test_gpu_vocab import BF16, F32, close, half_step, run_ce, run_distill

pytestmark = pytest.mark.gpu

# N of each first product: FMAs (fp32 tables), 32, 64 and 128 columns, tiles of pairs
NS = [5, 60, 100, 300]
TYPES = [(BF16, BF16, BF16, BF16), (BF16, BF16, F32, F32), (BF16, BF16, BF16, F32), (F32, F32, F32, F32), (BF16, F32, F32, F32), (F32, BF16, BF16, BF16)]


def logits(h, W, scale):
    return scale * (h.double() @ W.double().T)


def logit_errors(h, W, scale):
    """Of the worst logit of each row: d products in fp32 and pieces of the operands, as in the other tests' E."""
    return 2 * (h.shape[1] + 16) * 2.0 ** -23 * scale * (h.double().abs() @ W.double().abs().T).amax(1)


def check(dz, part, h, W, dh, dW, scale, rounded=1):
    """Gradients from dz [N, V] (64 bits), each entry of which may be off by `part`. rounded: operands besides dz's that a bf16
    gradient rounds."""
    h, W = h.double(), W.double()
    N, V = dz.shape
    tiny = 2.0 ** -125  # exponentials, pieces and products below the normal range are zero
    # an fp32 gradient's sums: 8 instructions of a k-block of 128, up to 32 rows by FMAs, and one addition a k-block or part
    add = lambda terms, g: (terms / 64 + 32 if g.dtype == F32 else terms + 16) * 2.0 ** -23  # noqa: E731
    if dh is not None:
        each = (2.0 ** -8 * (1 + rounded) if dh.dtype == BF16 else 2.0 ** -21) + add(V, dh)
        off = scale * ((part + each * (dz.abs() + part) + tiny) @ W.abs()) + tiny * V
        want = scale * (dz @ W)
        close(dh, want, off + half_step(dh.dtype) * (want.abs() + off), "grad_h")
    if dW is not None:
        each = (2.0 ** -8 * (1 + rounded) if dW.dtype == BF16 else 2.0 ** -20) + add(N, dW)
        off = scale * ((part + each * (dz.abs() + part) + tiny).T @ h.abs()) + tiny * N
        want = scale * (dz.T @ h)
        close(dW, want, off + half_step(dW.dtype) * (want.abs() + off), "grad_W")


def level(N, V, d, hdt, wdt, cuda):
    """Logits of 4000 and a little: whole numbers / 4, all products and sums exact."""
    gen = torch.Generator().manual_seed(N + V + d)
    W = torch.randint(-1, 2, (V, d), generator=gen).float()
    h = torch.randint(-1, 2, (N, d), generator=gen).float()
    W[:, 0] = 128.0
    h[:, 0] = 125.0
    t = torch.randint(0, V, (N,), generator=gen, dtype=torch.int32)
    return h.to(hdt).to(cuda), W.to(wdt).to(cuda), t.to(cuda), 0.25


@pytest.mark.parametrize("hdt,wdt,ghd,gwd", TYPES)
@pytest.mark.parametrize("N", NS)
@pytest.mark.parametrize("V,d", [(700, 64), (3000, 520)])
def test_weights_of_rows_whose_logits_are_all_large(cuda, N, V, d, hdt, wdt, ghd, gwd):
    # the differences are exact; lse itself is only known to 2^-24 of 4000, and no factor of the gradients may come of it
    h, W, t, scale = level(N, V, d, hdt, wdt, cuda)
    z = logits(h, W, scale)
    p = torch.softmax(z, 1)
    rel = 2.0 ** -22 * (2 * float(z.amax(1).sub(z.amin(1)).max()) + 80)
    ids = torch.stack([t, (t + 1) % V], 1).int().contiguous()
    u = torch.tensor([math.log(3.0), 0.0], device=cuda).repeat(N, 1)
    others = torch.ones(V, dtype=torch.bool, device=cuda)
    others[ids.flatten().long()] = False           # tokens that are no row's target
    dz = torch.where(others, 2 * p, 0.0)
    for dW in (run_ce(h, W, t, ghd, gwd, scale=scale, grad_scale=2.0)[3], run_distill(h, W, ids, u, ghd, gwd, scale=scale, grad_scale=2.0)[3]):
        check(dz, rel * dz, h, W, None, torch.where(others[:, None], dW, 0.0), scale)
