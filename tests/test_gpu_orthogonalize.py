"""pg_orthogonalize where its roundings could grow: matrices of few directions and of decaying
spectra, against the formulas in 64 bits and against the formulas rounded where the kernel rounds.

What is rounded: A and Bm = a I + b A + c A A to fp16 (half a step: 2^-11 of the entry) but for their
diagonals; X to the sum of two fp16 numbers (2^-22), the second of which the last step leaves out (2^-11,
times a); the result to bf16. A rounding of X lies in all singular directions and grows by a = 3.44 a
step where G has none (485-fold over five steps), so it has to start at 2^-22; one of A or Bm multiplies X,
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
    """The formulas with A, Bm and the two parts of X rounded to fp16 as the kernel holds them, and what that
    leaves of the diagonals of A and Bm."""
    a, b, c = coeffs
    outs = []
    for g in G.double():
        x = g if g.shape[0] <= g.shape[1] else g.T
        x = x / (torch.linalg.norm(x) + eps)
        for s in range(steps):
            hi = fp16_held(x)
            lo = fp16_held(x - hi) if s + 1 < steps else torch.zeros_like(x)
            exact = hi @ hi.T
            A = fp16_held(exact)
            left = exact.diagonal() - A.diagonal()
            exact = b * A + c * (A @ A) + torch.diag(a + left * (b + 2 * c * A.diagonal()))
            B = fp16_held(exact)
            ratio = (exact.diagonal() / B.diagonal())[:, None]
            x = ratio * (B @ (hi + lo)) if len(A) <= 128 else ratio * (B @ hi) + a * lo
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


@pytest.mark.parametrize("kind", ["gaussian", "rank11"])
@pytest.mark.parametrize("m,n", [(32, 984), (1400, 40), (40, 1400), (296, 1536), (1536, 296), (16, 4000)])
def test_sides_many_times_the_other(cuda, m, n, kind):
    # singular values near one another, where diagonals rounded to fp16 lose most: what the held forms add
    # stays below what rounding the result to bf16 does, and independent errors add in squares
    G = make(kind, 2, m, n, F32, cuda) if kind == "rank11" else gaussian(torch.Generator().manual_seed(m), 2, m, n, F32, cuda)
    out, ref = run_ortho(_pg(), G), ortho_reference(G, 5)
    assert rel(out, ref) <= math.sqrt(2.0) * rel(ref.to(BF16), ref)


def test_one_direction_per_matrix_of_a_batch(cuda):
    # the low parts of one matrix do not reach another
    G = torch.cat([make(k, 1, 200, 264, F32, cuda) for k in ("rank1", "decay3", "rank2", "rank4+0.01")])
    out = run_ortho(_pg(), G)
    want = ortho_reference(G, 5)
    for i in range(4):
        assert rel(out[i], want[i]) <= FORMULA, i


# From 4,194,304 values on, norm and scaling are launches of their own, with other blocks and shares.


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("b,m,n,shift", [(5, 2560, 1280, 0), (1, 2048, 2048, 0), (1, 2047, 2049, 0), (3, 1201, 1203, 0),
                                         (400, 104, 104, 0), (700, 79, 77, 0), (2, 1500, 1400, 1), (2, 1400, 1504, 4)])
def test_large_batches(cuda, b, m, n, shift, dtype):
    # 400 and 700 matrices: one part each, and blocks of the scaling that cross matrices; an odd n or an
    # address off by `shift` values: a column at a time
    assert b * m * n >= 4 << 20 or (b, m, n) == (1, 2047, 2049)  # one value short: the single launch
    pg = _pg()
    G = offset_view(gaussian(torch.Generator().manual_seed(b + m * n), b, m, n, dtype, cuda), shift)
    out = offset_view(torch.full((b, m, n), float("nan"), dtype=BF16, device=cuda), shift)
    ws = torch.full((pg.orthogonalize_workspace_size(b, m, n),), 0xA5, dtype=torch.uint8, device=cuda)
    pg.orthogonalize(G, out, ws)
    assert pg.device_error() == 0
    assert rel(out, held_reference(G)) <= SAME_PLACES
    assert rel(out, ortho_reference(G, 5)) <= FORMULA


@pytest.mark.parametrize("b,m,n", [(5, 1000, 1000), (3, 1201, 1203), (2, 300, 200), (1, 131, 129)])
def test_in_place(cuda, b, m, n):
    pg = _pg()
    G = gaussian(torch.Generator().manual_seed(b), b, m, n, BF16, cuda)
    want = run_ortho(pg, G)
    ws = torch.empty(pg.orthogonalize_workspace_size(b, m, n), dtype=torch.uint8, device=cuda)
    for _ in range(3):
        buf = G.clone()
        pg.orthogonalize(buf, buf, ws)
        assert torch.equal(buf, want)


def test_large_zero_nan_and_neighbours(cuda):
    pg = _pg()
    for n in (1000, 1001):
        G = gaussian(torch.Generator().manual_seed(8), 5, 1100, n, F32, cuda)
        G[1] = 0
        G[2, 3, 4] = math.nan
        G[3, 1099, n - 1] = math.inf
        out = run_ortho(pg, G)
        assert rel(out[0], ortho_reference(G[:1], 5)[0]) <= FORMULA
        assert bool((out[1] == 0).all())
        assert bool(out[2].isnan().all()) and bool(out[3].isnan().all())
        assert rel(out[4], ortho_reference(G[4:], 5)[0]) <= FORMULA


@pytest.mark.parametrize("std", [1e-30, 1e30])
def test_large_of_any_magnitude(cuda, std):
    G = gaussian(torch.Generator().manual_seed(9), 3, 1200, 1200, F32, cuda, std)
    out = run_ortho(_pg(), G, eps=0.0)
    assert rel(out, held_reference(G, eps=0.0)) <= SAME_PLACES


@pytest.mark.parametrize("b,m,n", [(2, 80, 120), (3, 1200, 1200)])
@pytest.mark.parametrize("std", [1e-44, 1e-39, 1e-37, 1e-33, 1e36, 3e37])
def test_norms_at_the_ends_of_fp32(cuda, b, m, n, std):
    # subnormal values; 2^10 / norm past fp32's range; norms past it of values in it. Small norms need eps = 0.
    G = gaussian(torch.Generator().manual_seed(9), b, m, n, F32, cuda, std)
    assert bool(G.isfinite().all()) and bool((G != 0).any())
    out = run_ortho(_pg(), G, eps=0.0)
    assert rel(out, held_reference(G, eps=0.0)) <= SAME_PLACES
    if std > 1:
        assert rel(run_ortho(_pg(), G), held_reference(G)) <= SAME_PLACES
