"""Digits that the vocabulary losses keep where a row's logits, or its weight, are far from one.

Tolerances. p = exp(z - lse) and 1 - p, the sum of the other tokens' exponentials over all, are sums and quotients of
exponentials of differences. An exponential has a relative error of 2^-22 from its own function, one of its argument's rounding
(2^-23 of the difference, twice: scale log2(e) has one too) and the sum of V terms 300 roundings; so a relative
REL = 2^-22 (2 difference + 80) of each of dz's parts, and of a loss as far as it comes of exponentials. On top comes twice what the
logits themselves are off, which is nothing where all their products and sums are whole numbers."""
import math

import pytest
import torch

from tests.test_gpu_vocab import BF16, F32, close, half_step, make, reference, run_ce, run_distill

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


@pytest.mark.parametrize("hdt,wdt,ghd,gwd", TYPES)
@pytest.mark.parametrize("N", NS)
@pytest.mark.parametrize("V,d", [(700, 64), (3000, 520)])
def test_rows_whose_logits_are_all_large(cuda, N, V, d, hdt, wdt, ghd, gwd):
    # the differences are exact, lse itself is only known to 2^-24 of 4000
    h, W, t, scale = level(N, V, d, hdt, wdt, cuda)
    z = logits(h, W, scale)
    lse = z.logsumexp(1)
    p = torch.softmax(z, 1)
    rel = 2.0 ** -22 * (2 * float(z.amax(1).sub(z.amin(1)).max()) + 80)
    one = torch.zeros_like(p).scatter(1, t.long()[:, None], 1.0)
    want = lse - z.gather(1, t.long()[:, None])[:, 0]
    loss, got, dh, dW = run_ce(h, W, t, ghd, gwd, scale=scale, grad_scale=2.0)
    for x in (loss, run_ce(h, W, t, scale=scale)[0]):
        close(x, want, rel + 2.0 ** -23 * want, "loss")
    close(got, lse, 2.0 ** -22 * lse, "lse")
    check(2 * (p - one), 2 * rel * p, h, W, dh, dW, scale)
    # a teacher of two tokens, weights 3 : 1
    ids = torch.stack([t, (t + 1) % V], 1).int().contiguous()
    u = torch.tensor([math.log(3.0), 0.0], device=cuda).repeat(N, 1)
    q = 0.75 * one + 0.25 * torch.zeros_like(p).scatter(1, ids[:, 1:].long(), 1.0)
    want = 0.75 * math.log(0.75) + 0.25 * math.log(0.25) - (q * (z - lse[:, None])).sum(1)
    loss, got, dh, dW = run_distill(h, W, ids, u, ghd, gwd, scale=scale, grad_scale=2.0)
    for x in (loss, run_distill(h, W, ids, u, scale=scale)[0]):
        close(x, want, rel + 2.0 ** -20 * (1 + want.abs()), "loss")
    close(got, lse, 2.0 ** -22 * lse, "lse")
    check(2 * (p - q), 2 * rel * p + 2 * 2.0 ** -21 * q, h, W, dh, dW, scale)


def confident(N, V, d, hdt, wdt, cuda, whole):
    """Rows whose target is 8 to 70 above the others, or (whole) 12 to 60 with logits that are whole numbers / 4."""
    gen = torch.Generator().manual_seed(N + V + d + whole)
    t = torch.randperm(V, generator=gen)[:N].to(torch.int32)
    if whole:
        W = (torch.rand(V, d, generator=gen) < 0.5).float() * 2 - 1      # <W_t, W_t> = d, others a few sqrt(d) at most
        h = torch.randint(1, 3, (N, 1), generator=gen).float() * W[t.long()]
        h = h + torch.randint(-1, 2, (N, d), generator=gen).float()
        scale = 0.25
    else:
        W = torch.randn(V, d, generator=gen) / math.sqrt(d)
        W = W.to(wdt).float()
        gap = 15 + 70 * torch.rand(N, 1, generator=gen)
        h = gap * W[t.long()] / (W[t.long()] ** 2).sum(1, keepdim=True) + 0.1 * torch.randn(N, d, generator=gen)
        scale = 1.0
    return h.to(hdt).to(cuda), W.to(wdt).to(cuda), t.to(cuda), scale


def exact_rows(h, W, t, scale):
    """z, softmax without the target's place, and one minus the target's p, without the difference of numbers near one."""
    z = logits(h, W, scale)
    at = t.long()[:, None]
    zt = z.gather(1, at)
    others = torch.exp(z - zt).scatter(1, at, 0.0)
    rest = others.sum(1, keepdim=True)             # (1 - p) / p
    return z, zt, others / (1 + rest), rest / (1 + rest), torch.log1p(rest)[:, 0]


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("hdt,wdt,ghd,gwd", TYPES)
@pytest.mark.parametrize("V,d", [(700, 128), (5003, 144)])
@pytest.mark.parametrize("N", NS)
def test_rows_that_are_sure_of_their_target(cuda, N, V, d, hdt, wdt, ghd, gwd, whole):
    h, W, t, scale = confident(N, V, d, hdt, wdt, cuda, whole)
    z, zt, p, missing, want = exact_rows(h, W, t, scale)
    assert float(missing.min()) < 1e-7 and (N < 60 or ((missing > 1e-20) & (missing < 1e-3)).sum() > N // 4)
    far = float((zt - z).abs().max())
    rel = 2.0 ** -22 * (2 * far + 80) + (0.0 if whole else 2 * logit_errors(h, W, scale))
    rel = rel if whole else rel[:, None]
    row = rel if whole else rel[:, 0]
    for zl in (0.0, 1e-3):
        lse = z.logsumexp(1)
        beta1 = 2 * zl * lse[:, None]              # beta - 1
        loss, got_lse, dh, dW = run_ce(h, W, t, ghd, gwd, scale=scale, z_loss=zl)
        forward = run_ce(h, W, t, scale=scale, z_loss=zl)
        lse_off = (0.0 if whole else logit_errors(h, W, scale)) + 2.0 ** -22 * (lse.abs() + 1)
        for got in (loss, forward[0]):
            if zl == 0:
                assert (got >= 0).all()
                close(got, want, row * want + 2.0 ** -125, "loss")
            else:
                close(got, want + zl * lse ** 2, row * want + zl * lse ** 2 * 2.0 ** -21 + 2 * zl * lse.abs() * lse_off + 2.0 ** -125, "loss")
        for got in (got_lse, forward[1]):
            close(got, lse, lse_off, "lse")
        dz = (1 + beta1) * p
        dz = dz.scatter(1, t.long()[:, None], beta1 * (1 - missing) - missing)
        b_off = 2 * zl * lse_off[:, None] + 2.0 ** -22 * beta1.abs()
        part = (rel * (1 + beta1) + b_off) * p
        part = part.scatter(1, t.long()[:, None], rel * missing + (rel * missing + 2.0 ** -22) * beta1.abs() + b_off)
        check(dz, part, h, W, dh, dW, scale)


@pytest.mark.parametrize("hdt,wdt,ghd,gwd", TYPES)
@pytest.mark.parametrize("N", NS)
@pytest.mark.parametrize("small", [1e-20, 1e-28])
def test_small_weights_of_rows_far_from_their_target(cuda, N, hdt, wdt, ghd, gwd, small):
    # logits up to 38 above the target's: sums below 2^57 of the target's term, which keep their reference
    V, d = 700, 64
    gen = torch.Generator().manual_seed(N)
    W = torch.randint(-1, 2, (V, d), generator=gen).float()
    h = torch.randint(-1, 2, (N, d), generator=gen).float()
    t = torch.randint(0, V, (N,), generator=gen, dtype=torch.int32)
    W[:, 0] = 64.0
    W[t.long(), 0] = 36.0
    h[:, 0] = 4.0                                  # 28 below the others, give or take a few
    h, W, t = h.to(hdt).to(cuda), W.to(wdt).to(cuda), t.to(cuda)
    scale = 0.25
    z = logits(h, W, scale)
    p = torch.softmax(z, 1)
    rel = 2.0 ** -22 * (2 * float(z.amax(1).sub(z.amin(1)).max()) + 80)
    one = torch.zeros_like(p).scatter(1, t.long()[:, None], 1.0)
    _, _, dh, dW = run_ce(h, W, t, ghd, gwd, scale=scale, grad_scale=small)
    check(small * (p - one), small * rel * (p + one), h, W, dh, dW, scale)
    # two rows of every three have ordinary weights
    weight = torch.where(torch.arange(N) % 3 == 0, small, 0.5).to(cuda)
    _, _, dh, dW = run_ce(h, W, t, ghd, gwd, scale=scale, weight=weight)
    g = weight.double()[:, None]
    check(g * (p - one), g * rel * (p + one), h, W, dh, dW, scale)


@pytest.mark.parametrize("hdt,wdt", [(F32, F32), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("N", NS + [9])
def test_fp32_values_beyond_the_largest_of_bf16(cuda, N, hdt, wdt):
    # finite, and multiplied by zeros: they must not become infinities
    h, W, t = make(N, N, 1200, 80, hdt, wdt, cuda)
    for x, y in ((W, h), (h, W)):
        if x.dtype == F32:
            hh, ww = h.clone(), W.clone()
            (ww if x is W else hh)[:, 5] = torch.finfo(F32).max
            (hh if x is W else ww)[:, 5] = 0.0
            plain_h, plain_w = hh.clone(), ww.clone()
            plain_h[:, 5] = plain_w[:, 5] = 0.0
            r = reference(plain_h, plain_w, t)
            loss, lse, _, _ = run_ce(hh, ww, t)
            E = torch.where(r["keep"], r["E"], 0.0)
            close(loss, r["loss"], 2 * E + 2.0 ** -22 * r["loss"].abs(), "loss")
            close(lse, r["lse"], E + 2.0 ** -23 * r["lse"].abs(), "lse")
            if x is W:  # (grad_W does not have W in it)
                _, _, _, dW = run_ce(hh, ww, t, None, F32)
                assert dW.isfinite().all()
                _, _, _, want = run_ce(plain_h, plain_w, t, None, F32)
                assert torch.equal(dW, want)
