"""The losses over the vocabulary against plain implementations in 64 bits: pg_vocab_ce, pg_vocab_distill and their
gradients.

Tolerances. A logit is an fp32 sum of d products: within (d + 16) 2^-23 of the sum of the products' magnitudes
(tensor cores may cut where others round; fp32 operands are three bf16 pieces, 2^-24 each, and three of the nine
products of pieces are left out, 2^-23 together: the 16). exp takes a relative error of 2^-22, of its argument's rounding
(2^-23 of the logits' size, twice) and a sum of the V terms 300 roundings at most (128 in a tile, then tiles spread over
16 warps). So lse and log p have E = 2 (d + 16) 2^-23 mag + 2^-22 (2 max|z| + 80). A gradient takes dz with p off by
E relative, a rounding of each operand it is made of (bf16: U, f h for grad_W and an fp32 W for grad_h, 2^-8 each; pieces:
2^-22 in all), fp32 sums ((terms + 16) 2^-23) and its own rounding.
"""
import math

import pytest
import torch

from tests._helpers import F32_TOL

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _pg():
    from hashed_head_gram_gb300 import pg
    return pg


def half_step(dtype):
    return 2.0 ** -8 if dtype == BF16 else 2.0 ** -24


def offset_view(t, shift):
    buf = torch.empty(t.numel() + shift, dtype=t.dtype, device=t.device)
    v = buf[shift:].view(t.shape)
    v.copy_(t)
    return v


def make(seed, N, V, d, hdt, wdt, dev, spread=1.0, K=0, pad=0.1):
    """Normed hidden states that lean towards their target's row, targets with padding, teacher lists."""
    gen = torch.Generator().manual_seed(seed)
    W = torch.randn(V, d, generator=gen) * (spread / math.sqrt(d))
    t = torch.randint(0, V, (N,), generator=gen, dtype=torch.int32)
    h = torch.randn(N, d, generator=gen) + torch.rand(N, 1, generator=gen) * 6 * W[t.long()] / spread ** 2
    gone = torch.rand(N, generator=gen) < pad
    t[gone] = torch.where(torch.rand(int(gone.sum()), generator=gen) < 0.5, -1, V).to(torch.int32)
    out = [h.to(hdt).to(dev), W.to(wdt).to(dev), t.to(dev)]
    if K:
        ids = torch.randint(0, V, (N, K), generator=gen, dtype=torch.int32)
        ids[torch.rand(N, K, generator=gen) < 0.1] = -1
        ids[gone] = V + 7
        u = torch.randn(N, K, generator=gen) * 3
        u[torch.rand(N, K, generator=gen) < 0.05] = float("-inf")
        out += [ids.to(dev), u.to(dev)]
    return out


def reference(h, W, target=None, ids=None, u=None, scale=1.0, T=1.0, z_loss=0.0, weight=None, grad_scale=1.0, grads=True):
    """loss, lse, dh, dW in 64 bits, and dz and the error that E leaves in it."""
    w32 = W.dtype == F32
    h, W = h.double(), W.double()
    s = scale / T
    z = s * (h @ W.T)
    N, V = z.shape
    mag = abs(s) * (h.abs() @ W.abs().T).amax(1)
    lse = torch.logsumexp(z, 1)
    q = torch.zeros_like(z)
    if ids is None:
        keep = (target >= 0) & (target < V)
        at = torch.nonzero(keep)[:, 0]
        q[at, target[at].long()] = 1.0
        ent = torch.zeros(N, dtype=torch.float64, device=z.device)
    else:
        there = (ids >= 0) & (ids < V)
        u = torch.where(there, u.double() / T, -math.inf)
        keep = (u > -math.inf).any(1)
        p = torch.softmax(torch.where(keep[:, None], u, 0.0), 1)
        p = torch.where(there & keep[:, None], p, 0.0)
        q.scatter_add_(1, torch.where(there, ids, 0).long(), p)
        ent = torch.where(p > 0, p * torch.log(torch.where(p > 0, p, 1.0)), 0.0).sum(1)
    loss = torch.where(keep, ent - (q * z).nan_to_num().sum(1) + lse + z_loss * lse * lse, 0.0)
    lse_out = torch.where(keep, lse, 0.0)
    E = 2 * (h.shape[1] + 16) * 2.0 ** -23 * mag + 2.0 ** -22 * (2 * z.abs().amax(1) + 80)
    if ids is not None:  # the teacher's own softmax in fp32
        E = E + 2.0 ** -22 * (4 + torch.where(u > -math.inf, u.abs(), 0.0).amax(1))
    r = dict(loss=loss, lse=lse_out, E=E, keep=keep, w32=w32)
    if grads:
        g = grad_scale * s * keep.double()
        if weight is not None:
            g = g * weight.double()
        beta = 1 + 2 * z_loss * lse
        prob = torch.softmax(z, 1)
        dz = torch.where(keep[:, None], g[:, None] * (beta[:, None] * prob - q), 0.0)
        off = torch.where(keep[:, None], (g.abs() * E)[:, None] * (beta.abs()[:, None] * prob + q * (ids is not None)), 0.0)
        # exponentials below 2^-126 of the row's reference, which is at most its sum, are zero, as are such pieces; and
        # pieces of dz below 2^-126 where U is dz
        off = torch.where(keep[:, None], off + 2.0 ** -125 * (1 + g.abs()[:, None]), off)
        hk = torch.where(keep[:, None], h, 0.0)
        r.update(dh=dz @ W, dW=dz.T @ hk, dz=dz, off=off, h=hk, W=W, g=float(g.abs().max()))
    return r


def close(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float(((got.double() - want).abs() / tol)[bad].max())} of the tolerance"


def distance(got, want):
    return float((got.double() - want).norm())


def check_values(r, loss, lse, z_loss=0.0):
    E = torch.where(r["keep"], r["E"], 0.0)
    close(lse, r["lse"], E + 2.0 ** -23 * r["lse"].abs(), "lse")
    close(loss, r["loss"], E * (2 + 2 * abs(z_loss) * r["lse"].abs()) + 2.0 ** -22 * r["loss"].abs(), "loss")


def check_grads(r, dh, dW, old=None):
    dz, off, W, h = r["dz"], r["off"], r["W"], r["h"]
    N, V = dz.shape
    # Independent roundings add in squares: of k uniform ones, 2^-8 at most each, the sum's root mean square is
    # sqrt(k) 2^-8 / sqrt(3). That is an average: over 21 entries of dz (3 x 7) a sum of three goes past 2^-8, its
    # mean, about every other time, so the norms are looked at where a few thousand entries take part
    many = N * V >= 4096 and min(N, V) >= 32
    if dh is not None:
        each = (1 + r["w32"]) * half_step(BF16) if dh.dtype == BF16 else 2.0 ** -22
        tol = (off + each * (dz.abs() + off)) @ W.abs() + (V + 16) * 2.0 ** -23 * (dz.abs() @ W.abs())
        tol = tol + V * 2.0 ** -126 * max(1.0, r["g"])  # products below the normal range are zero
        tol = tol + half_step(dh.dtype) * (r["dh"].abs() + tol)
        close(dh, r["dh"], tol, "grad_h")
        # two roundings (bf16; of an fp32 W a third). What E leaves in p comes on
        # top: dz = g (beta p - 1) at a target with p near 1 is the difference of two numbers near g, so an
        # error of E in p is E / |beta p - 1| of dz (a vocabulary of one token: p = 1, beta - 1 = 2 z_loss lse)
        assert not many or distance(dh, r["dh"]) <= (2.0 ** -8 if dh.dtype == BF16 else F32_TOL) * float(r["dh"].norm()) + float((off @ W.abs()).norm())
        assert (dh[~r["keep"]] == 0).all()
    if dW is not None:
        each = 2 * half_step(BF16) if dW.dtype == BF16 else 2.0 ** -21
        tol = (off + each * (dz.abs() + off)).T @ h.abs() + (N + 16) * 2.0 ** -23 * (dz.abs().T @ h.abs())
        want = r["dW"] if old is None else r["dW"] + old.double()
        chunk = 0.0 if old is None else half_step(F32) * old.double().abs()
        tol = tol + chunk + N * 2.0 ** -126
        tol = tol + half_step(dW.dtype) * (want.abs() + tol) + 2.0 ** -126
        close(dW, want, tol, "grad_W")
        if old is None:  # three roundings
            assert not many or distance(dW, r["dW"]) <= (2.0 ** -8 if dW.dtype == BF16 else F32_TOL) * float(r["dW"].norm()) + float((off.T @ h.abs()).norm())


def run_ce(h, W, t, ghd=None, gwd=None, shift=0, weight=None, accumulate=None, **kw):
    """vocab_ce, or with gradient dtypes vocab_ce_grad: loss, lse, grad_h, grad_W. Outputs and workspace start as NaN."""
    pg = _pg()
    N, d = h.shape
    V, dev = W.shape[0], h.device
    nan = lambda shape, t: offset_view(torch.full(shape, float("nan"), dtype=t, device=dev), shift)  # noqa: E731
    loss, lse = nan((N,), F32), nan((N,), F32)
    hd, wd = pg.dtype_code(h.dtype), pg.dtype_code(W.dtype)
    if ghd is None and gwd is None:
        ws = torch.full((pg.vocab_ce_workspace_size(N, V, d, hd, wd),), 0xFF, dtype=torch.uint8, device=dev)
        pg.vocab_ce(h, W, t, loss, ws, lse=lse, **kw)
        return loss, lse, None, None
    gh = None if ghd is None else nan((N, d), ghd)
    gw = None if gwd is None else nan((V, d), gwd) if accumulate is None else accumulate
    size = pg.vocab_ce_grad_workspace_size(N, V, d, hd, wd, None if ghd is None else pg.dtype_code(ghd),
                                           None if gwd is None else pg.dtype_code(gwd))
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=dev)
    pg.vocab_ce_grad(h, W, t, loss, gh, gw, ws, lse=lse, row_weight=weight, accumulate=accumulate is not None, **kw)
    assert pg.device_error() == 0
    return loss, lse, gh, gw


def run_distill(h, W, ids, u, ghd=None, gwd=None, weight=None, **kw):
    pg = _pg()
    N, d = h.shape
    V, K, dev = W.shape[0], ids.shape[1], h.device
    nan = lambda shape, t: torch.full(shape, float("nan"), dtype=t, device=dev)  # noqa: E731
    loss, lse = nan((N,), F32), nan((N,), F32)
    hd, wd = pg.dtype_code(h.dtype), pg.dtype_code(W.dtype)
    if ghd is None and gwd is None:
        ws = torch.full((pg.vocab_distill_workspace_size(N, V, d, K, hd, wd),), 0xFF, dtype=torch.uint8, device=dev)
        pg.vocab_distill(h, W, ids, u, loss, ws, lse=lse, **kw)
        return loss, lse, None, None
    gh = None if ghd is None else nan((N, d), ghd)
    gw = None if gwd is None else nan((V, d), gwd)
    size = pg.vocab_distill_grad_workspace_size(N, V, d, K, hd, wd, None if ghd is None else pg.dtype_code(ghd),
                                                None if gwd is None else pg.dtype_code(gwd))
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=dev)
    pg.vocab_distill_grad(h, W, ids, u, loss, gh, gw, ws, lse=lse, row_weight=weight, **kw)
    assert pg.device_error() == 0
    return loss, lse, gh, gw


# up to 128 rows the first product is another kernel (of 32, 64 and 128 columns); d = 1500: sums in groups
SHAPES = [(1, 1, 1), (1, 1000, 64), (3, 7, 5), (8, 4096, 256), (33, 999, 200), (64, 2050, 136), (100, 1300, 1500), (128, 641, 96),
          (129, 641, 96), (200, 300, 72), (256, 256, 128), (257, 513, 130), (300, 1023, 515), (300, 2000, 1500), (700, 5000, 96),
          (31, 70001, 40)]


@pytest.mark.parametrize("hdt,wdt", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("N,V,d", SHAPES)
def test_ce(cuda, N, V, d, hdt, wdt):
    h, W, t = make(N + V + d, N, V, d, hdt, wdt, cuda)
    r = reference(h, W, t, scale=0.8, z_loss=1e-3, grads=False)
    loss, lse, _, _ = run_ce(h, W, t, scale=0.8, z_loss=1e-3)
    assert _pg().device_error() == 0
    check_values(r, loss, lse, 1e-3)


@pytest.mark.parametrize("hdt,wdt,ghd,gwd", [(BF16, BF16, BF16, BF16), (F32, F32, F32, F32), (BF16, F32, BF16, F32),
                                             (F32, BF16, BF16, BF16), (BF16, BF16, F32, F32), (BF16, BF16, BF16, F32)])
@pytest.mark.parametrize("N,V,d", SHAPES)
def test_ce_grad(cuda, N, V, d, hdt, wdt, ghd, gwd):
    h, W, t = make(2 * N + V + d, N, V, d, hdt, wdt, cuda)
    weight = torch.rand(N, generator=torch.Generator().manual_seed(5)).to(cuda) * 2 - 0.3
    r = reference(h, W, t, scale=1.2, z_loss=1e-3, weight=weight, grad_scale=1.0 / N)
    loss, lse, dh, dW = run_ce(h, W, t, ghd, gwd, weight=weight, scale=1.2, z_loss=1e-3, grad_scale=1.0 / N)
    check_values(r, loss, lse, 1e-3)
    check_grads(r, dh, dW)


@pytest.mark.parametrize("hdt,wdt,ghd,gwd", [(BF16, BF16, BF16, BF16), (F32, F32, F32, F32), (BF16, F32, BF16, F32)])
@pytest.mark.parametrize("N,V,d,K", [(1, 1, 1, 1), (1, 1000, 64, 20), (3, 7, 5, 6), (200, 300, 72, 33), (257, 513, 130, 100),
                                     (40, 2000, 64, 50), (100, 97, 1500, 30), (300, 600, 1500, 64), (700, 5000, 96, 256), (31, 70001, 40, 3)])
@pytest.mark.parametrize("T", [1.0, 2.5])
def test_distill(cuda, N, V, d, K, T, hdt, wdt, ghd, gwd):
    h, W, _, ids, u = make(3 * N + V + d, N, V, d, hdt, wdt, cuda, K=K)
    if hdt == BF16:
        u = u.to(BF16)
    r = reference(h, W, ids=ids, u=u, scale=1.1, T=T, grad_scale=1.0 / N)
    loss, lse, _, _ = run_distill(h, W, ids, u, scale=1.1, temperature=T)
    check_values(r, loss, lse)
    loss, lse, dh, dW = run_distill(h, W, ids, u, ghd, gwd, scale=1.1, temperature=T, grad_scale=1.0 / N)
    check_values(r, loss, lse)
    check_grads(r, dh, dW)


# Up to 8 rows an fp32 W is multiplied in fp32: four values of a row at a time, or one where d is odd or W
# starts on 4 bytes alone; more segments and parts than warps; last segments and parts of one row. Beside them more rows, which
# take W in pieces
@pytest.mark.parametrize("hdt,ghd,gwd", [(F32, F32, F32), (F32, BF16, BF16), (F32, BF16, F32), (BF16, F32, None), (BF16, BF16, None), (F32, None, F32),
                                         (BF16, None, None)])
@pytest.mark.parametrize("N,V,d,shift", [(1, 1025, 4, 0), (1, 1025, 64, 1), (5, 80000, 260, 0), (5, 40000, 260, 3), (8, 20481, 129, 0), (9, 1153, 2052, 0),
                                         (7, 30000, 65, 0), (8, 30001, 520, 0), (6, 1100, 1021, 0), (17, 20000, 68, 0), (128, 3000, 320, 2)])
def test_few_rows_of_an_fp32_table(cuda, N, V, d, shift, hdt, ghd, gwd):
    h, W, t = make(5 * N + V + d, N, V, d, hdt, F32, cuda)
    W = offset_view(W, shift)
    r = reference(h, W, t, scale=0.9, z_loss=1e-3, grad_scale=1.0 / N)
    loss, lse, dh, dW = run_ce(h, W, t, ghd, gwd, scale=0.9, z_loss=1e-3, **({} if ghd is None and gwd is None else {"grad_scale": 1.0 / N}))
    check_values(r, loss, lse, 1e-3)
    check_grads(r, dh, dW)


def test_few_rows_of_an_fp32_table_lists_and_large_logits(cuda):
    # tokens far above the target (rows that change their reference) and lists over all of the table's tiles
    for N, V, d in [(3, 5000, 100), (8, 21000, 72), (5, 90001, 33), (128, 2049, 130)]:
        h, W, t, ids, u = make(N + V, N, V, d, F32, F32, cuda, K=100)
        r = reference(h, W, ids=ids, u=u, scale=1.1, T=2.0, grad_scale=1.0 / N)
        loss, lse, dh, dW = run_distill(h, W, ids, u, F32, F32, scale=1.1, temperature=2.0, grad_scale=1.0 / N)
        check_values(r, loss, lse)
        check_grads(r, dh, dW)
        r = reference(40 * h, W, t, grad_scale=1.0 / N)
        loss, lse, dh, dW = run_ce(40 * h, W, t, F32, F32, grad_scale=1.0 / N)
        check_values(r, loss, lse)
        check_grads(r, dh, dW)


@pytest.mark.parametrize("hdt,ghd,gwd", [(BF16, BF16, BF16), (F32, F32, F32)])
@pytest.mark.parametrize("N,V,d", [(20011, 300, 72), (9000, 1024, 256), (4097, 64, 33)])
def test_many_rows_of_a_small_table(cuda, N, V, d, hdt, ghd, gwd):
    # grad_W's few tiles are cut along the rows
    h, W, t = make(N, N, V, d, hdt, hdt, cuda)
    r = reference(h, W, t, grad_scale=1.0 / N)
    loss, lse, dh, dW = run_ce(h, W, t, ghd, gwd, grad_scale=1.0 / N)
    check_values(r, loss, lse)
    check_grads(r, dh, dW)


def gathered(dz, p, z, h):
    """What the cuts of tensor-core sums come to in dW, as a norm: one a k-block of 128 for the logits, one a 64 rows for dW."""
    # Each addition (of 16 products) cuts below 2^-23 of the sum, always to one side, so logits are off by 8 2^-23 |z| at most and
    # their errors add up over the rows, the targets' too, which the row's sum has from there
    cut = 8 * 2.0 ** -23 * z.abs()
    first = p * (cut - (p * cut).sum(1, keepdim=True)) / z.shape[0]
    # and dW's sums of four additions by 4 2^-23 of each
    second = sum((dz[i:i + 64].T @ h[i:i + 64]).abs() for i in range(0, z.shape[0], 64))
    return float((first.T @ h).norm()) + 4 * 2.0 ** -23 * float(second.norm())


@pytest.mark.parametrize("N,V,d", [(20011, 600, 760), (11708, 604, 1200), (3001, 1100, 2500)])
def test_an_fp32_table_gradient_gathers_little_of_what_sums_cut(cuda, N, V, d):
    # states that lean to their targets by up to 12 logits, a few targets in most rows
    gen = torch.Generator().manual_seed(N)
    W = (torch.randn(V, d, generator=gen) / math.sqrt(d)).to(BF16)
    t = (torch.rand(N, generator=gen) ** 3 * V).to(torch.int32)
    h = (torch.randn(N, d, generator=gen) + torch.rand(N, 1, generator=gen) * 12 * W[t.long()].float()).to(BF16)
    h, W, t = h.to(cuda), W.to(cuda), t.to(cuda)
    r = reference(h, W, t, grad_scale=1.0 / N)
    loss, lse, dh, dW = run_ce(h, W, t, BF16, F32, grad_scale=1.0 / N)
    z = h.double() @ W.double().T
    # beside the cuts roundings of 2^-21 or so of each of dz's values, which add in squares, and of the sums in fp32
    each = 2.0 ** -21 * float(((r["dz"] ** 2).T @ h.double() ** 2).sqrt().norm()) + 2.0 ** -21 * float(r["dW"].norm())
    assert distance(dW, r["dW"]) <= gathered(r["dz"], torch.softmax(z, 1), z, h.double()) + each


@pytest.mark.parametrize("ghd,gwd,accumulate", [(F32, BF16, False), (F32, BF16, True), (F32, F32, False), (F32, F32, True), (None, F32, False),
                                                (F32, None, False)])
def test_rows_in_chunks(cuda, ghd, gwd, accumulate):
    # three pieces of 70,001 columns: 4864 rows are 2 GiB, so the rows come in two chunks
    N, V, d = 6000, 70001, 40
    h, W, t = make(11, N, V, d, F32, F32, cuda, pad=0.3)
    r = reference(h, W, t, grad_scale=0.01)
    old = None
    if accumulate:
        old = torch.randn(V, d, generator=torch.Generator().manual_seed(3)).to(gwd).to(cuda) * 0.01
    loss, lse, dh, dW = run_ce(h, W, t, ghd, gwd, grad_scale=0.01, accumulate=None if old is None else old.clone())
    check_values(r, loss, lse)
    check_grads(r, dh, dW, old)


def test_many_chunks_of_the_forward_call(cuda):
    N, V, d = 40000, 900, 24
    h, W, t = make(12, N, V, d, BF16, BF16, cuda)
    r = reference(h, W, t, grads=False)
    loss, lse, _, _ = run_ce(h, W, t)
    check_values(r, loss, lse)
