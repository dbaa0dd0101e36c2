"""The training calls against plain implementations in 64 bits: pg_embed, pg_embed_grad,
pg_lookup_grad (rows and signs from the CPU oracle) and pg_orthogonalize.

Tolerances. A sum of c fp32 terms carries at most (c + 2) roundings of 2^-24 of the sum of
magnitudes (the additions, the scale and the store); a bf16 result half a bf16 step more.
"""
import dataclasses
import math

import numpy as np
import pytest
import torch

from hashed_head_gram_gb300 import workloads as W
from oracle import oracle as orc
from tests._helpers import canon_tensor, shrink_table

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _pg():
    from hashed_head_gram_gb300 import pg
    return pg


def half_step(dtype):
    return 2.0 ** -8 if dtype == BF16 else 2.0 ** -24


def assert_sums(got, ref, mag, counts, out_dtype, old=None):
    """got against the fp64 sums `ref`, whose terms' magnitudes add up to `mag`."""
    tol = (counts + 2) * 2.0 ** -24 * mag
    if old is not None:
        tol = tol + 2.0 ** -24 * (ref.abs() + old.abs())
    tol = tol + half_step(out_dtype) * (ref.abs() + tol)
    bad = (got.double() - ref).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} elements off"


def offset_view(t, shift):
    """The same values at an address `shift` elements past an allocation's start."""
    buf = torch.empty(t.numel() + shift, dtype=t.dtype, device=t.device)
    v = buf[shift:].view(t.shape)
    v.copy_(t)
    return v


def make_ids(gen, n, vocab, kind, dev):
    if kind == "same":
        t = torch.full((n,), vocab // 3, dtype=torch.int32)
    elif kind == "padding":
        t = torch.full((n,), -1, dtype=torch.int32)
    elif kind == "skewed":  # one ID takes a third of the batch, the rest are spread
        t = torch.randint(0, vocab, (n,), generator=gen, dtype=torch.int32)
        t[torch.rand(n, generator=gen) < 0.33] = 1
    else:
        t = torch.randint(0, vocab, (n,), generator=gen, dtype=torch.int32)
        bad = torch.rand(n, generator=gen)
        t[bad < 0.05] = -5
        t[bad > 0.95] = vocab + 3
    return t.to(dev)


def embed_rows(tokens, cmap, vocab, rows):
    t = tokens.cpu().long()
    ok = (t >= 0) & (t < vocab)
    t = torch.where(ok, t, 0)
    if cmap is not None:
        t = cmap.cpu().long()[t]
    ok &= t < rows
    return torch.where(ok, t, -1)


# ---------------------------------------------------------------------------------- embed


@pytest.mark.parametrize("table_dtype", [F32, BF16])
@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("N,d,shift", [(1, 1, 0), (7, 33, 0), (300, 96, 0), (300, 96, 1), (300, 96, 4), (5, 2560, 0), (129, 1032, 0),
                                       (64, 1025, 0), (40001, 24, 0), (39999, 13, 0)])
def test_embed(cuda, table_dtype, out_dtype, N, d, shift):
    pg = _pg()
    gen = torch.Generator().manual_seed(N * 1000 + d)
    vocab, rows = 900, 700
    tokens = make_ids(gen, N, vocab, "mixed", cuda)
    cmap = torch.randint(0, rows + 20, (vocab,), generator=gen, dtype=torch.int32).to(cuda)  # some past the table
    table = offset_view(torch.randn(rows, d, generator=gen).to(table_dtype).to(cuda), shift)
    out = offset_view(torch.full((N, d), float("nan"), dtype=out_dtype, device=cuda), shift)
    err = torch.zeros(1, dtype=torch.int32, device=cuda)
    scale = math.sqrt(d)
    pg.embed(tokens, table, out, vocab, scale=scale, canon_map=cmap, err_index=err)
    at = embed_rows(tokens, cmap, vocab, rows)
    ref = torch.where(at[:, None] >= 0, table.cpu()[at.clamp(min=0)].double() * float(np.float32(scale)), 0.0)
    got = out.cpu().double()
    assert bool(((got - ref).abs() <= (2.0 ** -24 + half_step(out_dtype)) * 1.01 * ref.abs()).all())
    bad = torch.nonzero(at < 0)
    assert err.item() == (int(bad[0]) if len(bad) else -1)


def test_embed_keeps_infinities_and_nan(cuda):
    pg = _pg()
    table = torch.tensor([[math.inf, -math.inf, math.nan, 0.0] * 2], device=cuda)
    out = torch.empty(2, 8, device=cuda)
    pg.embed(torch.tensor([0, -1], dtype=torch.int32, device=cuda), table, out, 1, scale=2.0)
    assert torch.equal(out[0].isnan(), table[0].isnan()) and torch.equal(out[0].isinf(), table[0].isinf())
    assert bool((out[1] == 0).all())  # padding takes nothing from row 0


# ----------------------------------------------------------------------------- embed_grad


def run_embed_grad(pg, tokens, grad, out, vocab, scale, cmap=None, accumulate=False, err=None, stream=None):
    ws = torch.empty(pg.embed_grad_workspace_size(tokens.numel(), *out.shape), dtype=torch.uint8, device=out.device)
    ws.fill_(0xA5)  # scratch: whatever is there
    pg.embed_grad(tokens, grad, out, vocab, ws, scale=scale, accumulate=accumulate, canon_map=cmap, err_index=err,
                  stream=stream)


def check_embed_grad(cuda, N, d, vocab, rows, kind, grad_dtype, out_dtype, accumulate=False, shift=0, canon=True, seed=0):
    pg = _pg()
    gen = torch.Generator().manual_seed(N * 31 + d + seed)
    tokens = make_ids(gen, N, vocab, kind, cuda)
    cmap = torch.randint(0, rows + (rows + 9) // 10, (vocab,), generator=gen, dtype=torch.int32).to(cuda) if canon else None
    grad = offset_view(torch.randn(N, d, generator=gen).to(grad_dtype).to(cuda), shift)
    old = torch.randn(rows, d, generator=gen).to(out_dtype).to(cuda)
    out = offset_view(old, shift)
    err = torch.zeros(1, dtype=torch.int32, device=cuda)
    scale = 1.7
    run_embed_grad(pg, tokens, grad, out, vocab, scale, cmap, accumulate, err)
    assert pg.device_error() == 0
    at = embed_rows(tokens, cmap, vocab, rows)
    keep = (at >= 0).to(cuda)
    at = at.to(cuda)
    ref = torch.zeros(rows, d, dtype=torch.float64, device=cuda)
    mag, counts = torch.zeros_like(ref), torch.zeros(rows, 1, dtype=torch.float64, device=cuda)
    ref.index_add_(0, at[keep], grad[keep].double())
    mag.index_add_(0, at[keep], grad[keep].double().abs())
    counts.index_add_(0, at[keep], torch.ones(int(keep.sum()), 1, dtype=torch.float64, device=cuda))
    s = float(np.float32(scale))
    if accumulate:
        untouched = counts[:, 0] == 0
        assert torch.equal(out[untouched].view(torch.uint8), old[untouched].view(torch.uint8))
        assert_sums(out, ref * s + old.double(), mag * s, counts, out_dtype, old.double())
    else:
        assert_sums(out, ref * s, mag * s, counts, out_dtype)
    bad = torch.nonzero(at < 0)
    assert err.item() == (int(bad[0]) if len(bad) else -1)


@pytest.mark.parametrize("grad_dtype,out_dtype", [(F32, F32), (BF16, F32), (BF16, BF16), (F32, BF16)])
@pytest.mark.parametrize("N,d", [(1, 8), (1, 1), (37, 33), (513, 96), (4097, 40)])
def test_embed_grad_types_and_sizes(cuda, N, d, grad_dtype, out_dtype):
    check_embed_grad(cuda, N, d, 900, 700, "mixed", grad_dtype, out_dtype)


@pytest.mark.parametrize("kind", ["same", "padding", "skewed", "mixed"])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("N,d,rows", [(20000, 16, 5000), (3000, 264, 77), (70001, 8, 120000)])
def test_embed_grad_distributions(cuda, kind, accumulate, N, d, rows):
    check_embed_grad(cuda, N, d, rows + 100, rows, kind, BF16, F32, accumulate, canon=False)


def test_embed_grad_unaligned_and_one_row(cuda):
    check_embed_grad(cuda, 2500, 96, 900, 700, "mixed", BF16, F32, shift=1)
    check_embed_grad(cuda, 2500, 96, 900, 700, "mixed", F32, BF16, shift=3, accumulate=True)
    check_embed_grad(cuda, 2500, 24, 3, 1, "skewed", F32, F32, canon=False)
    check_embed_grad(cuda, 40000, 2, 3, 2, "mixed", F32, F32, canon=False)


@pytest.mark.parametrize("shift", [0, 1])
def test_embed_grad_widest_rows(cuda, shift):
    check_embed_grad(cuda, 20, 1 << 20, 4, 3, "mixed", F32, BF16, shift=shift)


def test_embed_grad_of_no_tokens(cuda):
    pg = _pg()
    out = torch.ones(5, 8, device=cuda)
    none = torch.empty(0, dtype=torch.int32, device=cuda)
    pg.embed_grad(none, torch.empty(0, 8, device=cuda), out, 5, None, accumulate=True)
    assert bool((out == 1).all())
    pg.embed_grad(none, torch.empty(0, 8, device=cuda), out, 5, None)
    assert bool((out == 0).all())


def test_embed_grad_padding_takes_no_infinity(cuda):
    pg = _pg()
    grad = torch.ones(4, 8, device=cuda)
    grad[1] = math.inf
    grad[2] = math.nan
    out = torch.empty(6, 8, device=cuda)
    run_embed_grad(pg, torch.tensor([2, -1, 6, 2], dtype=torch.int32, device=cuda), grad, out, 6, 1.0)
    assert bool((out[2] == 2).all()) and out.sum().item() == 16


def test_embed_grad_is_the_adjoint_of_embed(cuda):
    # <embed(E), g> = <E, embed_grad(g)> for a linear operator; integers, so every sum is exact
    pg = _pg()
    gen = torch.Generator().manual_seed(4)
    N, d, vocab = 3001, 40, 500
    tokens = make_ids(gen, N, vocab, "mixed", cuda)
    E = torch.randint(-8, 9, (vocab, d), generator=gen).float().to(cuda)
    g = torch.randint(-8, 9, (N, d), generator=gen).float().to(cuda)
    out, grad = torch.empty(N, d, device=cuda), torch.empty(vocab, d, device=cuda)
    pg.embed(tokens, E, out, vocab, scale=2.0)
    run_embed_grad(pg, tokens, g, grad, vocab, 2.0)
    assert (out.double() * g.double()).sum().item() == (E.double() * grad.double()).sum().item()


# ---------------------------------------------------------------------------- lookup_grad


def run_lookup_grad(pg, desc, tokens, grad, n, r, out_dtype, cmap=None, err=None, stream=None, shift=0):
    dev = grad.device
    rows = torch.full((n,), 7, dtype=torch.int32, device=dev)
    out = offset_view(torch.full((n, r), float("nan"), dtype=out_dtype, device=dev), shift)
    count = torch.full((1,), -9, dtype=torch.int32, device=dev)
    ws = torch.full((pg.lookup_grad_workspace_size(desc, tokens.numel()),), 0xA5, dtype=torch.uint8, device=dev)
    pg.lookup_grad(desc, tokens, grad, rows, out, count, ws, canon_map=cmap, err_index=err, stream=stream)
    return rows, out, count


def check_lookup_grad(cuda, spec, tokens, vocab, cmap, grad_dtype, out_dtype, shift=0):
    pg = _pg()
    gen = torch.Generator().manual_seed(tokens.size + spec.r)
    N, H = tokens.size, 1 if spec.mode == W.MODE_FLAT else spec.K
    O, r = len(spec.orders), spec.r
    n = N * O * H
    grad = offset_view(torch.randn(N, spec.e_width, generator=gen).to(grad_dtype).to(cuda), shift)
    desc = pg.table_desc(spec, vocab)
    rows, out, count = run_lookup_grad(pg, desc, torch.from_numpy(tokens).to(cuda), grad, n, r, out_dtype,
                                       canon_tensor(cmap, cuda), shift=shift)
    assert pg.device_error() == 0
    _, ref_rows, signs, bad = orc.index(spec, tokens, cmap, vocab)
    assert bad == -1
    ref_rows = ref_rows.reshape(-1).astype(np.int64)
    bits = np.unpackbits(np.ascontiguousarray(signs.reshape(n, -1)).astype("<u8").view(np.uint8), axis=1, bitorder="little")[:, :r]
    g = grad.cpu().double().numpy()
    g = np.repeat(g[:, None], O, 1).reshape(n, r) if spec.mode == W.MODE_FLAT else g.reshape(n, r)
    uniq, inv, cnt = np.unique(ref_rows, return_inverse=True, return_counts=True)
    inv = torch.from_numpy(inv.reshape(-1))
    ref = torch.zeros(len(uniq), r, dtype=torch.float64).index_add_(0, inv, torch.from_numpy(np.where(bits, -g, g)))
    mag = torch.zeros_like(ref).index_add_(0, inv, torch.from_numpy(np.abs(g)))
    assert count.item() == len(uniq)
    got_rows = rows.cpu().numpy().view(np.uint32)
    assert np.array_equal(got_rows[:len(uniq)], uniq.astype(np.uint32)) and bool((got_rows[len(uniq):] == 0xFFFFFFFF).all())
    out = out.cpu()
    assert_sums(out[:len(uniq)], ref, mag, torch.from_numpy(cnt)[:, None].double(), out_dtype)
    assert bool((out[len(uniq):] == 0).all())


SPECS = {
    "pagegram": lambda: shrink_table(W.make_workload(2).tables[0]),
    "engram80": lambda: shrink_table(W.make_workload(5).tables[0]),
    "flat768": lambda: shrink_table(W.make_workload(3).tables[1]),
    "pagegram-fp32": lambda: W.make_workload(1).tables[0],
    "nf4": lambda: shrink_table(W.make_workload(4).tables[0]),
    "orders1-4": lambda: W.TableSpec("o4", W.MODE_ENGRAM, K=3, S=1, r=24, row_dtype=0, orders=[1, 2, 3, 4], hash_seed=5,
                                     rows=[[101, 97, 89], [4001, 3989, 53], [1, 2, 3], [70001, 7, 11]]),
    "odd-width": lambda: W.TableSpec("odd", W.MODE_PAGEGRAM, K=5, S=3, r=13, row_dtype=0, orders=[2, 4], pages=[41, 2003],
                                     hash_seed=99),
    "wide-heads": lambda: W.TableSpec("wide", W.MODE_ENGRAM, K=2, S=1, r=600, row_dtype=0, orders=[2], rows=[[211, 199]],
                                      hash_seed=3),
    "flat-odd": lambda: W.TableSpec("flat-odd", W.MODE_FLAT, K=1, S=1, r=131, row_dtype=0, orders=[1, 2, 3],
                                    rows=[[50], [60], [70]], hash_seed=8),
    "32-heads": lambda: W.TableSpec("h32", W.MODE_PAGEGRAM, K=16, S=2, r=8, row_dtype=1, orders=[2, 3], pages=[300, 301],
                                    hash_seed=12),
    "one-row": lambda: W.TableSpec("one", W.MODE_FLAT, K=1, S=1, r=16, row_dtype=0, orders=[2], rows=[[1]], hash_seed=1),
}


@pytest.mark.parametrize("name", list(SPECS))
@pytest.mark.parametrize("B,L", [(1, 1), (3, 37), (2, 700)])
@pytest.mark.parametrize("grad_dtype,out_dtype", [(F32, F32), (BF16, F32), (BF16, BF16)])
def test_lookup_grad(cuda, name, B, L, grad_dtype, out_dtype):
    rng = np.random.default_rng(B * 100 + L)
    vocab = 300
    tokens = np.minimum(rng.zipf(1.3, (B, L)) - 1, vocab - 1).astype(np.int32)
    cmap = rng.integers(0, 250, vocab).astype(np.uint32) if L != 37 else None
    check_lookup_grad(cuda, SPECS[name](), tokens, vocab, cmap, grad_dtype, out_dtype)


@pytest.mark.parametrize("name", ["pagegram", "engram80", "flat768", "odd-width"])
def test_lookup_grad_of_one_repeated_token(cuda, name):
    tokens = np.full((2, 3000), 17, np.int32)  # every position past the window reads the same rows
    check_lookup_grad(cuda, SPECS[name](), tokens, 300, None, BF16, F32)


def test_lookup_grad_many_reads_and_large_row_numbers(cuda):
    # 600,000 reads over 2^25 + rows: every block of the sort, three digits
    spec = W.TableSpec("large", W.MODE_ENGRAM, K=4, S=1, r=8, row_dtype=1, orders=[2, 3], hash_seed=77,
                       rows=[W.largest_primes(6_000_000, 4)] * 2)
    rng = np.random.default_rng(3)
    tokens = np.minimum(rng.zipf(1.15, (25, 3000)) - 1, 49999).astype(np.int32)
    check_lookup_grad(cuda, spec, tokens, 50000, None, F32, F32)
    # rows past 2^31: the keys' top bit counts
    huge = dataclasses.replace(spec, K=2, rows=[[1_500_000_007, 1_000_000_007], [900_000_011, 800_000_011]])
    check_lookup_grad(cuda, huge, tokens[:2], 50000, None, F32, F32)


@pytest.mark.parametrize("name", ["pagegram", "orders1-4", "flat-odd"])
def test_lookup_grad_shares_of_several_tiles(cuda, name):
    # more reads than the sort's blocks hold at once (152 * 8192)
    spec = dataclasses.replace(SPECS[name](), r=8)
    reads = len(spec.orders) * (1 if spec.mode == W.MODE_FLAT else spec.K)
    L = 2_700_000 // reads // 3
    rng = np.random.default_rng(17)
    tokens = np.minimum(rng.zipf(1.2, (3, L)) - 1, 299).astype(np.int32)
    check_lookup_grad(cuda, spec, tokens, 300, None, F32, F32)


def test_embed_grad_shares_of_several_tiles(cuda):
    check_embed_grad(cuda, 1_400_003, 8, 70_000, 60_000, "mixed", BF16, F32)
    check_embed_grad(cuda, 1_300_000, 8, 300, 200, "skewed", F32, F32, accumulate=True, canon=False)


def test_offsets_past_32_bits(cuda):
    # tables of more than 2^32 elements: only the rows looked at are checked
    pg = _pg()
    rows, d = 70_000, 65_600
    at = torch.tensor([0, 1, 65_472, 65_473, 69_999, 33_000, 69_999], dtype=torch.int32, device=cuda)
    table = torch.empty(rows, d, dtype=BF16, device=cuda)
    gen = torch.Generator(device=cuda).manual_seed(1)
    vals = torch.randn(len(at), d, generator=gen, device=cuda).to(BF16)
    table[at.long()] = vals
    out = torch.empty(len(at), d, dtype=BF16, device=cuda)
    pg.embed(at, table, out, rows, scale=2.0)
    assert torch.equal(out, table[at.long()] * 2)
    grad = torch.randn(len(at), d, generator=gen, device=cuda).to(BF16)
    ws = torch.empty(pg.embed_grad_workspace_size(len(at), rows, d), dtype=torch.uint8, device=cuda)
    pg.embed_grad(at, grad, table, rows, ws)
    want = grad.clone()
    want[4] = want[6] = (grad[4].float() + grad[6].float()).to(BF16)
    assert torch.equal(table[at.long()], want)
    rest = torch.ones(rows, dtype=torch.bool, device=cuda)
    rest[at.long()] = False
    for part in torch.nonzero(rest)[:, 0].split(8000):
        assert not table[part].any()


def test_lookup_grad_unaligned(cuda):
    rng = np.random.default_rng(8)
    tokens = rng.integers(0, 300, (2, 90)).astype(np.int32)
    for shift in (1, 4):
        check_lookup_grad(cuda, SPECS["pagegram"](), tokens, 300, None, BF16, F32, shift=shift)


def test_lookup_grad_reads_bad_tokens_as_id_0(cuda):
    pg = _pg()
    spec = SPECS["pagegram"]()
    desc = pg.table_desc(spec, 300)
    good = torch.randint(0, 300, (2, 50), dtype=torch.int32, generator=torch.Generator().manual_seed(1))
    good[1, 7] = 0
    bad = good.clone()
    bad[1, 7] = 300
    grad = torch.randn(100, 1024, generator=torch.Generator().manual_seed(2)).to(cuda)
    err = torch.zeros(1, dtype=torch.int32, device=cuda)
    a = run_lookup_grad(pg, desc, good.to(cuda), grad, 1600, 64, F32, err=err)
    assert err.item() == -1
    b = run_lookup_grad(pg, desc, bad.to(cuda), grad, 1600, 64, F32, err=err)
    assert err.item() == 57
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_lookup_grad_of_no_tokens(cuda):
    pg = _pg()
    desc = pg.table_desc(SPECS["pagegram"](), 300)
    z = lambda *s, dt=F32: torch.empty(*s, dtype=dt, device=cuda)  # noqa: E731
    count = torch.full((1,), 5, dtype=torch.int32, device=cuda)
    pg.lookup_grad(desc, z(0, 5, dt=torch.int32), z(0, 1024), z(0, dt=torch.int32), z(0, 64), count, None)
    assert count.item() == 0


@pytest.mark.parametrize("name", ["pagegram-fp32", "orders1-4", "flat768"])
def test_lookup_grad_matches_differences_of_the_lookup(cuda, name):
    # f(T) = <lookup(T), g> is linear in T: f(T + D) - f(T) = <grad, D>; integers keep it exact
    pg = _pg()
    spec = dataclasses.replace(SPECS[name](), row_dtype=0)
    gen = torch.Generator().manual_seed(6)
    desc = pg.table_desc(spec, 300)
    tokens = torch.randint(0, 300, (2, 150), dtype=torch.int32, generator=gen).to(cuda)
    T = torch.randint(-8, 9, (spec.table_rows, spec.r), generator=gen).float().to(cuda)
    D = torch.randint(-8, 9, (spec.table_rows, spec.r), generator=gen).float().to(cuda)
    g = torch.randint(-8, 9, (300, spec.e_width), generator=gen).float().to(cuda)

    def f(table):
        e = torch.empty(300, spec.e_width, device=cuda)
        pg.gather_sign_concat(desc, tokens, table, e, pg.F32)
        return (e.double() * g.double()).sum().item()

    n = 300 * len(spec.orders) * (1 if spec.mode == W.MODE_FLAT else spec.K)
    rows, grads, count = run_lookup_grad(pg, desc, tokens, g, n, spec.r, F32)
    c = count.item()
    want = (grads[:c].double() * D[rows[:c].long()].double()).sum().item()
    assert f(T + D) - f(T) == want


def test_gradients_are_reproducible_and_follow_their_stream(cuda):
    pg = _pg()
    spec = SPECS["pagegram"]()
    desc = pg.table_desc(spec, 300)
    gen = torch.Generator().manual_seed(11)
    tokens = make_ids(gen, 6000, 300, "skewed", cuda).view(4, 1500)
    grad = torch.randn(6000, 1024, generator=gen).to(cuda)
    first = run_lookup_grad(pg, desc, tokens, grad, 96000, 64, F32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        late = grad * 1.0                     # made on the side stream
        second = run_lookup_grad(pg, desc, tokens, late, 96000, 64, F32)
        out = torch.empty(300, 1024, device=cuda)
        run_embed_grad(pg, tokens.view(-1), late, out, 300, 1.0)
    side.synchronize()
    for x, y in zip(first, second):
        assert torch.equal(x, y)
    again = torch.empty(300, 1024, device=cuda)
    run_embed_grad(pg, tokens.view(-1), grad, again, 300, 1.0)
    assert torch.equal(out, again)


# -------------------------------------------------------------------------- orthogonalize

COEFFS = (3.4445, -4.7750, 2.0315)


def ortho_reference(G, steps, coeffs=COEFFS, eps=1e-7, scale=1.0, hold=None):
    """The formulas in 64 bits; `hold` rounds X, A and a I + b A + c A A where the kernel stores them."""
    a, b, c = coeffs
    hold = hold or (lambda x: x)
    outs = []
    for g in G.double():
        x = g if g.shape[0] <= g.shape[1] else g.T
        x = hold(x / (torch.linalg.norm(x) + eps))
        for s in range(steps):
            A = hold(x @ x.T)
            x = hold(a * torch.eye(len(A), dtype=A.dtype, device=A.device) + b * A + c * (A @ A)) @ x
            if s + 1 < steps:
                x = hold(x)
        outs.append(scale * (x if g.shape[0] <= g.shape[1] else x.T))
    return torch.stack(outs)


def fp16_held(x):
    return (x * 1024).half().double() / 1024


def run_ortho(pg, G, **kw):
    b, m, n = G.shape if G.dim() == 3 else (1, *G.shape)
    ws = torch.full((pg.orthogonalize_workspace_size(b, m, n),), 0xA5, dtype=torch.uint8, device=G.device)
    out = torch.full(G.shape, float("nan"), dtype=BF16, device=G.device)
    pg.orthogonalize(G, out, ws, **kw)
    assert pg.device_error() == 0
    return out


def gaussian(gen, b, m, n, dtype, dev, std=1e-3):
    return (torch.randn(b, m, n, generator=gen) * std).to(dtype).to(dev)


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


# Against the formulas rounded to fp16 at the same places: what differs is the order of fp32
# sums (a rounding to fp16 moves by one step where a sum lands next to a boundary: a small
# share of the values, 2^-11 each) and the bf16 result: half a step, 2^-8, per value at most.
SAME_PLACES = 2.0 ** -8
# Against the formulas in 64 bits: each of the 5 steps stores three matrices with relative
# error 2^-11 at most; the map p(s) = a s + b s^3 + c s^5 stretches an error by at most 4
# where it stretches the values by up to 3.44, so an error of step k ends at most
# (4 / 3.44)^(5 - k) as large, relative to the result; with the coefficients' 4-fold weight of
# A: 4 * 2^-11 * (1 + 1.16 + .. + 1.16^4) = 1.4e-2, and the bf16 result's 2^-8.
FORMULA = 1.4e-2 + 2.0 ** -8


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("b,m,n", [(1, 1, 1), (1, 1, 300), (2, 200, 1), (3, 7, 5), (1, 64, 64), (2, 128, 256), (1, 256, 1024),
                                   (2, 129, 130), (1, 131, 515), (3, 515, 131), (1, 768, 1024), (2, 640, 320),
                                   (1, 1000, 777), (6, 520, 1030), (3, 1001, 1111), (3, 1111, 1001), (1, 2560, 1280),
                                   (5, 1040, 640)])
def test_orthogonalize(cuda, b, m, n, dtype):
    pg = _pg()
    G = gaussian(torch.Generator().manual_seed(m * n), b, m, n, dtype, cuda)
    out = run_ortho(pg, G)
    assert rel(out, ortho_reference(G, 5, hold=fp16_held)) <= SAME_PLACES
    assert rel(out, ortho_reference(G, 5)) <= FORMULA


def test_orthogonalize_singular_values(cuda):
    # known singular vectors: five steps bring singular values in [0.02, 1] into about one
    pg = _pg()
    gen = torch.Generator().manual_seed(5)
    u, _ = torch.linalg.qr(torch.randn(200, 200, generator=gen, dtype=torch.float64))
    v, _ = torch.linalg.qr(torch.randn(300, 200, generator=gen, dtype=torch.float64))
    s = torch.logspace(0, -1.5, 200, dtype=torch.float64)
    G = (u * s @ v.T).float().to(cuda)
    out = run_ortho(pg, G)
    sv = torch.linalg.svdvals(out.double())
    assert 0.6 < sv.min().item() and sv.max().item() < 1.3
    assert rel(out, ortho_reference(G[None], 5)[0]) <= FORMULA


@pytest.mark.parametrize("steps,coeffs,scale", [(1, COEFFS, 1.0), (2, (1.5, -0.5, 0.0), 0.2), (8, (2.0, -1.5, 0.5), 3.0)])
def test_orthogonalize_steps_coefficients_and_scale(cuda, steps, coeffs, scale):
    pg = _pg()
    G = gaussian(torch.Generator().manual_seed(steps), 2, 96, 160, F32, cuda)
    out = run_ortho(pg, G, steps=steps, coeffs=coeffs, scale=scale)
    assert rel(out, ortho_reference(G, steps, coeffs, scale=scale, hold=fp16_held)) <= SAME_PLACES


@pytest.mark.parametrize("std", [1e-30, 1e-12, 1e12, 1e30])
def test_orthogonalize_of_any_magnitude(cuda, std):
    # squares of these values leave fp32's range
    pg = _pg()
    G = gaussian(torch.Generator().manual_seed(9), 1, 80, 120, F32, cuda, std)
    out = run_ortho(pg, G, eps=0.0)
    assert rel(out, ortho_reference(G, 5, eps=0.0, hold=fp16_held)) <= SAME_PLACES


def test_orthogonalize_zero_nan_and_neighbours(cuda):
    pg = _pg()
    G = gaussian(torch.Generator().manual_seed(2), 4, 70, 90, F32, cuda)
    G[1] = 0
    G[2, 3, 4] = math.nan
    G[3, 5, 6] = math.inf
    out = run_ortho(pg, G)
    alone = run_ortho(pg, G[:1].contiguous())
    assert torch.equal(out[0], alone[0])           # a matrix does not see its neighbours
    assert bool((out[1] == 0).all())
    assert bool(out[2].isnan().all()) and bool(out[3].isnan().all())


def test_orthogonalize_in_place_reproducible_and_graphs(cuda):
    pg = _pg()
    G = gaussian(torch.Generator().manual_seed(3), 2, 300, 200, BF16, cuda)
    first = run_ortho(pg, G)
    assert torch.equal(first, run_ortho(pg, G))
    ws = torch.empty(pg.orthogonalize_workspace_size(2, 300, 200), dtype=torch.uint8, device=cuda)
    buf = G.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pg.orthogonalize(buf, buf, ws)             # out is G itself
    buf.copy_(G)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(buf, first)


def test_gradients_in_a_graph(cuda):
    pg = _pg()
    spec = SPECS["engram80"]()
    desc = pg.table_desc(spec, 300)
    gen = torch.Generator().manual_seed(21)
    tokens = make_ids(gen, 2000, 300, "skewed", cuda).view(2, 1000)
    grad = torch.randn(2000, 1280, generator=gen).to(BF16).to(cuda)
    want = run_lookup_grad(pg, desc, tokens, grad, 32000, 80, F32)
    rows, out, count = torch.empty_like(want[0]), torch.empty_like(want[1]), torch.empty_like(want[2])
    table = torch.empty(300, 1280, device=cuda)
    ws = torch.empty(pg.lookup_grad_workspace_size(desc, 2000), dtype=torch.uint8, device=cuda)
    ws2 = torch.empty(pg.embed_grad_workspace_size(2000, 300, 1280), dtype=torch.uint8, device=cuda)
    expect = torch.empty_like(table)
    run_embed_grad(pg, tokens.view(-1), grad, expect, 300, 0.5)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pg.lookup_grad(desc, tokens, grad, rows, out, count, ws)
        pg.embed_grad(tokens.view(-1), grad, table, 300, ws2, scale=0.5)
    for _ in range(2):
        rows.zero_(), out.zero_(), count.zero_(), table.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(rows, want[0]) and torch.equal(out, want[1]) and torch.equal(count, want[2])
        assert torch.equal(table, expect)


# ------------------------------------------------------------------------------ together


def test_training_example_learns(cuda):
    # embedding, lookup, projection, both gradients and the orthogonalised update in one loop
    from examples.train_memory import train
    losses = train(steps=30, n_tokens=4096).tolist()
    assert all(math.isfinite(x) for x in losses)
    assert losses[-1] < 0.5 * losses[0], losses
    assert _pg().device_error() == 0
