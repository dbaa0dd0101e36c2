"""pg_orthogonalize where its roundings could grow: matrices of few directions and of decaying
spectra, against the formulas in 64 bits and against the formulas rounded where the kernel rounds.

What is rounded: A and Bm = a I + b A + c A A to fp16 (half a step: 2^-11 of the entry); X to the sum
of two fp16 numbers (2^-22), the second of which the last step leaves out (2^-11, times a); the
result to bf16. A rounding of X lies in all singular directions and grows by a = 3.44 a step
where G has none (485-fold over five steps), so it has to start at 2^-22; one of A or Bm multiplies X,
lies only where X has directions, and stays what it is relative to the result.
"""
import math

import pytest
import torch

from tests.test_gpu_training import BF16, COEFFS, F32, _pg, fp16_held, gaussian, offset_view, ortho_reference, rel, run_ortho

pytestmark = pytest.mark.gpu

# Against the formulas rounded at the same places: the order of fp32 sums, which moves a small share of
# the fp16 values by one step of 2^-11, and the bf16 result, 2^-8 a value at most.
SAME_PLACES = 2.0 ** -8
# Against the formulas in 64 bits, per step and relative to the result: A, made of hi alone, and Bm
# with 2^-11 each, A weighing up to 4 times through Bm's coefficients, so 5 * 2^-11 where all errors
# add up, over five steps; the last step's X a * 2^-11; the bf16 result 2^-8.
FORMULA = 5 * 5 * 2.0 ** -11 + 3.4445 * 2.0 ** -11 + 2.0 ** -8


def held_reference(G, steps=5, coeffs=COEFFS, eps=1e-7, scale=1.0):
    """The formulas with A, Bm and the two parts of X rounded to fp16 as the kernel holds them."""
    a, b, c = coeffs
    outs = []
    for g in G.double():
        x = g if g.shape[0] <= g.shape[1] else g.T
        x = x / (torch.linalg.norm(x) + eps)
        for s in range(steps):
            hi = fp16_held(x)
            lo = fp16_held(x - hi) if s + 1 < steps else torch.zeros_like(x)
            A = fp16_held(hi @ hi.T)
            B = fp16_held(a * torch.eye(len(A), dtype=A.dtype, device=A.device) + b * A + c * (A @ A))
            x = B @ hi + (B @ lo if len(A) <= 128 else a * lo)
        outs.append(scale * (x if g.shape[0] <= g.shape[1] else x.T))
    return torch.stack(outs)


def make(kind, b, m, n, dtype, dev):
    gen = torch.Generator().manual_seed(m * 3 + n)
    randn = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    if kind.startswith("rank"):
        r = int(kind[4:].split("+")[0])
        G = randn(b, m, r) @ randn(b, r, n)
        if "+" in kind:  # noise of that share of the norm
            e = randn(b, m, n)
            G = G + e * (float(kind.split("+")[1]) * G.norm() / e.norm())
    else:  # singular values over that many decades
        p = min(m, n)
        u, _ = torch.linalg.qr(randn(b, m, p))
        v, _ = torch.linalg.qr(randn(b, n, p))
        G = u * torch.logspace(0, -float(kind[5:]), p, dtype=torch.float64) @ v.mT
    return (G * 1e-3).to(dtype).to(dev)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", ["rank1", "rank4", "rank11", "rank4+0.01", "rank4+1e-4", "decay3", "decay6"])
@pytest.mark.parametrize("b,m,n", [(1, 24, 24), (2, 100, 128), (1, 300, 128), (1, 131, 515), (1, 256, 1024), (1, 512, 512),
                                   (2, 300, 200), (1, 1280, 2560), (2, 1500, 1400)])
def test_few_directions(cuda, b, m, n, kind, dtype):
    G = make(kind, b, m, n, dtype, cuda)
    out = run_ortho(_pg(), G)
    assert rel(out, held_reference(G)) <= SAME_PLACES
    assert rel(out, ortho_reference(G, 5)) <= FORMULA


@pytest.mark.parametrize("m,n", [(90, 128), (128, 90), (130, 700), (700, 130)])
@pytest.mark.parametrize("steps", [1, 2, 3, 4])
def test_few_directions_in_few_steps(cuda, m, n, steps):
    # which steps write and read the low part of X
    G = make("rank3", 2, m, n, F32, cuda)
    out = run_ortho(_pg(), G, steps=steps, scale=0.5)
    assert rel(out, held_reference(G, steps, scale=0.5)) <= SAME_PLACES
    assert rel(out, ortho_reference(G, steps, scale=0.5)) <= FORMULA


def test_one_direction_per_matrix_of_a_batch(cuda):
    # the low parts of one matrix do not reach another
    G = torch.cat([make(k, 1, 200, 264, F32, cuda) for k in ("rank1", "decay3", "rank2", "rank4+0.01")])
    out = run_ortho(_pg(), G)
    want = ortho_reference(G, 5)
    for i in range(4):
        assert rel(out[i], want[i]) <= FORMULA, i
