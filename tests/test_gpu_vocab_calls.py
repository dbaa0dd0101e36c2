"""The vocabulary losses where their calls are unusual: rows without targets and what lies in them, logits far above the
targets', lists of every kind, streams, graphs, shared and separate workspaces, odd addresses, offsets past 32 bits."""
import math

import pytest
import torch

from tests.test_gpu_vocab import (BF16, F32, check_grads, check_values, half_step, make, offset_view, reference, run_ce,
                                  run_distill, _pg)

pytestmark = pytest.mark.gpu

# N of each first product: 32, 64 and 128 columns, tiles of pairs
NS = [5, 60, 100, 300]


@pytest.mark.parametrize("N", NS)
@pytest.mark.parametrize("hdt", [BF16, F32])
def test_padded_rows_may_hold_anything(cuda, N, hdt):
    h, W, t = make(N, N, 700, 80, hdt, hdt, cuda, pad=0.3)
    t[:2] = torch.tensor([-1, 700], device=cuda)
    gone = (t < 0) | (t >= 700)
    r = reference(h, W, t, z_loss=1e-3, grad_scale=0.1)
    for fill in (float("nan"), float("inf"), -float("inf"), torch.finfo(hdt).max, torch.finfo(hdt).min):
        h2 = h.clone()
        h2[gone] = fill
        loss, lse, _, _ = run_ce(h2, W, t, z_loss=1e-3)
        check_values(r, loss, lse, 1e-3)
        for gwd in (hdt, F32):
            loss, lse, dh, dW = run_ce(h2, W, t, hdt, gwd, z_loss=1e-3, grad_scale=0.1)
            check_values(r, loss, lse, 1e-3)
            check_grads(r, dh, dW)


@pytest.mark.parametrize("N", NS)
def test_no_targets_at_all(cuda, N):
    h, W, t = make(N, N, 700, 80, BF16, BF16, cuda)
    h.fill_(float("nan"))
    err = torch.full((1,), 77, dtype=torch.int32, device=cuda)
    loss, lse, dh, dW = run_ce(h, W, torch.full_like(t, -1), BF16, F32, err_index=err)
    assert err.item() == 0
    for x in (loss, lse, dh, dW):
        assert (x == 0).all()
    ids = torch.full((N, 4), 700, dtype=torch.int32, device=cuda)
    loss, lse, dh, dW = run_distill(h, W, ids, torch.zeros(N, 4, device=cuda), F32, BF16)
    for x in (loss, lse, dh, dW):
        assert (x == 0).all()


@pytest.mark.parametrize("N", NS)
def test_rows_of_weight_zero(cuda, N):
    # no gradient whatever they hold; their losses are still told
    h, W, t = make(N + 1, N, 700, 80, BF16, BF16, cuda, pad=0.0)
    weight = torch.rand(N, generator=torch.Generator().manual_seed(1)).to(cuda) + 0.5
    weight[::3] = 0
    h2 = h.clone()
    h2[::3] = float("nan")
    h2[3::6] = float("inf")
    r = reference(torch.where(weight[:, None] > 0, h, 0.0), W, t, weight=weight)
    keep = weight > 0
    r["keep"] = keep
    for gwd in (BF16, F32):
        loss, _, dh, dW = run_ce(h2, W, t, BF16, gwd, weight=weight)
        assert loss[~keep].isnan().all()
        assert (loss[keep].double() - r["loss"][keep]).abs().max() <= 1e-4
        check_grads(r, dh, dW)


def test_infinities_in_a_row_with_a_target_reach_it_alone(cuda):
    h, W, t = make(9, 300, 700, 80, BF16, BF16, cuda, pad=0.0)
    h2 = h.clone()
    h2[7, 3] = float("inf")
    loss, lse, dh, _ = run_ce(h2, W, t, BF16, None)
    want_loss, want_lse, want_dh, _ = run_ce(h, W, t, BF16, None)
    for got, want in ((loss, want_loss), (lse, want_lse), (dh, want_dh)):
        assert got[7].isnan().any()
        keep = torch.arange(300, device=cuda) != 7
        assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("N,V,d", [(5, 700, 80), (100, 1000, 80), (300, 1000, 80), (300, 40, 16), (300, 3000, 1500)])
@pytest.mark.parametrize("dt,ghd,gwd", [(BF16, BF16, BF16), (F32, F32, F32), (BF16, BF16, F32)])
@pytest.mark.parametrize("scale", [40.0, -60.0, 400.0])
def test_logits_far_above_the_targets(cuda, N, V, d, dt, ghd, gwd, scale):
    # sums beyond 2^57 of the target's term in some segments of most rows: those change their reference
    h, W, t = make(N + V, N, V, d, dt, dt, cuda, pad=0.1)
    t = torch.where(t >= 0, (t + 3) % V, t)  # away from the rows that h leans towards
    r = reference(h, W, t, scale=scale, grad_scale=1.0 / N)
    above = (r["lse"] - (scale * (h.double() @ W.double().T)).gather(1, t.clamp(0, V - 1).long()[:, None])[:, 0])[r["keep"]]
    assert N < 100 or (above > 60).sum() >= 3
    loss, lse, dh, dW = run_ce(h, W, t, ghd, gwd, scale=scale, grad_scale=1.0 / N)
    check_values(r, loss, lse)
    check_grads(r, dh, dW)
    ids, u = torch.stack([t, (t + 1) % V], 1).int().contiguous(), torch.zeros(N, 2, device=cuda)
    r = reference(h, W, ids=ids, u=u, scale=scale, grad_scale=1.0 / N)
    loss, lse, dh, dW = run_distill(h, W, ids, u, ghd, gwd, scale=scale, grad_scale=1.0 / N)
    check_values(r, loss, lse)
    check_grads(r, dh, dW)


@pytest.mark.parametrize("N", NS)
def test_lists_of_every_kind(cuda, N):
    V, d, K = 700, 80, 40
    h, W, _, ids, u = make(N + 2, N, V, d, BF16, BF16, cuda, K=K, pad=0.0)
    low = torch.finfo(F32).min
    ids[0] = 5                       # one token, all places
    ids[1, 1:] = ids[1, :1]          # twice and more, weights that add up
    u[2] = low                       # the type's lowest everywhere: even weights
    u[3, 1:] = low                   # but for one
    ids[4] = -1                      # nothing listed
    if N > 5:
        u[5] = -math.inf             # nothing of weight
        ids[6, 1:] = V               # one place
        u[7, 1:] = -math.inf         # one weight
        ids[8] = torch.arange(K, dtype=torch.int32) * 17  # ascending
        ids[9] = ids[8].flip(0)
        u[10] *= 1e4                 # a weight of one, the others 0
    r = reference(h, W, ids=ids, u=u, T=0.7, grad_scale=1.0)
    loss, lse, _, _ = run_distill(h, W, ids, u, temperature=0.7)
    # (u of 1e4 is a matter of the teacher's softmax: equal values' differences of 2^-23 of 1e4 and more are real)
    check_values(r, loss, lse)
    err = torch.full((1,), 77, dtype=torch.int32, device=cuda)
    loss, lse, dh, dW = run_distill(h, W, ids, u, BF16, BF16, temperature=0.7, err_index=err)
    check_values(r, loss, lse)
    check_grads(r, dh, dW)
    bad = ((ids < 0) | (ids >= V)).any(1).nonzero()
    assert err.item() == int(bad[0])
    run_distill(h, W, ids.clamp(0, V - 1), u, err_index=err)
    assert err.item() == -1


@pytest.mark.parametrize("N,V,K", [(5, 64, 200), (100, 300, 120), (300, 64, 256), (600, 200, 100), (300, 3000, 256)])
@pytest.mark.parametrize("d", [40, 1500])
def test_dense_lists(cuda, N, V, K, d):
    # most tokens of a tile are listed, many of them more than once
    h, W, _, ids, u = make(N + V + K, N, V, d, BF16, BF16, cuda, K=K)
    r = reference(h, W, ids=ids, u=u, T=2.0)
    loss, lse, _, _ = run_distill(h, W, ids, u, temperature=2.0)
    check_values(r, loss, lse)
    loss, lse, dh, dW = run_distill(h, W, ids, u, BF16, F32, temperature=2.0)
    check_values(r, loss, lse)
    check_grads(r, dh, dW)


def test_nan_and_infinite_teacher_logits_stay_in_their_row(cuda):
    h, W, _, ids, u = make(31, 300, 700, 80, BF16, BF16, cuda, K=8, pad=0.0)
    ids = ids.clamp(min=0)
    want = run_distill(h, W, ids, u, BF16, None)
    u2 = u.clone()
    u2[11, 2], u2[20, 0] = float("nan"), float("inf")
    got = run_distill(h, W, ids, u2, BF16, None)
    keep = torch.ones(300, dtype=torch.bool, device=cuda)
    keep[[11, 20]] = False
    for g, w in zip(got[:3], want[:3]):
        assert torch.equal(g[keep], w[keep])
    assert got[0][[11, 20]].isnan().all() and got[2][[11, 20]].isnan().any(1).all()


def test_a_list_of_one_is_cross_entropy(cuda):
    h, W, t = make(17, 333, 1000, 96, BF16, BF16, cuda)
    a = run_ce(h, W, t, BF16, BF16, scale=0.9)
    b = run_distill(h, W, t[:, None].contiguous(), torch.linspace(-3, 3, 333, device=cuda)[:, None].contiguous(), BF16, BF16, scale=0.9)
    for x, y in zip(a, b):
        close = (x.double() - y.double()).abs()
        assert (close <= 2.0 ** -7 * (x.double().abs() + 1e-3 * x.double().abs().max())).all()


@pytest.mark.parametrize("op", ["ce", "distill"])
def test_gradients_are_differences(cuda, op):
    N, V, d = 6, 50, 12
    h, W, t, ids, u = make(3, N, V, d, F32, F32, cuda, K=5, pad=0.2)
    weight = torch.linspace(0.5, 1.5, N, device=cuda)

    def total(hh, WW):
        if op == "ce":
            loss = reference(hh, WW, t, z_loss=0.01, grads=False)["loss"]
        else:
            loss = reference(hh, WW, ids=ids, u=u, T=1.7, grads=False)["loss"]
        return float((loss * weight.double()).sum())

    if op == "ce":
        _, _, dh, dW = run_ce(h, W, t, F32, F32, weight=weight, z_loss=0.01)
    else:
        _, _, dh, dW = run_distill(h, W, ids, u, F32, F32, weight=weight, temperature=1.7)
    step = 1e-5  # differences in 64 bits: off by step^2 times third derivatives, a few 1e-10
    h, W = h.double(), W.double()
    for x, g in ((h, dh), (W, dW)):
        for i in range(0, x.numel(), 7):
            keep = x.view(-1)[i].item()
            x.view(-1)[i] = keep + step
            up = total(h, W)
            x.view(-1)[i] = keep - step
            down = total(h, W)
            x.view(-1)[i] = keep
            assert abs((up - down) / (2 * step) - float(g.view(-1)[i])) <= 2e-5


@pytest.mark.parametrize("N,V,d", [(5, 700, 80), (300, 700, 80), (130, 641, 33), (60, 300, 36)])
@pytest.mark.parametrize("ghd,gwd", [(BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("shift", [1, 3, 4])
def test_odd_addresses(cuda, N, V, d, ghd, gwd, shift):
    h, W, t = make(N + d, N, V, d, F32, F32, cuda)
    h, W, t = offset_view(h, shift), offset_view(W, shift), offset_view(t, shift)
    weight = offset_view(torch.rand(N, generator=torch.Generator().manual_seed(d)).to(cuda), shift)
    r = reference(h, W, t, weight=weight)
    loss, lse, dh, dW = run_ce(h, W, t, ghd, gwd, shift=shift, weight=weight)
    check_values(r, loss, lse)
    check_grads(r, dh, dW)
    if d % 8:  # bf16 that is copied first
        h, W = offset_view(h.to(BF16), shift), offset_view(W.to(BF16), shift)
        r = reference(h, W, t, weight=weight)
        loss, lse, dh, dW = run_ce(h, W, t, ghd, gwd, shift=shift, weight=weight)
        check_values(r, loss, lse)
        check_grads(r, dh, dW)


@pytest.mark.parametrize("N,V,d,gd", [(5, 700, 80, BF16), (100, 641, 33, F32), (300, 700, 80, BF16), (300, 641, 33, F32), (1000, 300, 40, F32)])
def test_nothing_else_is_written(cuda, N, V, d, gd):
    pg = _pg()
    h, W, t = make(N, N, V, d, BF16, BF16, cuda)
    size = pg.vocab_ce_grad_workspace_size(N, V, d, 1, 1, pg.dtype_code(gd), pg.dtype_code(gd))
    guard = 512
    bufs = {k: torch.full((n + 2 * guard,), 7.5, dtype=dt, device=cuda) for k, n, dt in
            [("loss", N, F32), ("lse", N, F32), ("gh", N * d, gd), ("gw", V * d, gd)]}
    ws = torch.full((size + 2 * guard,), 0x5A, dtype=torch.uint8, device=cuda)
    view = lambda k, shape: bufs[k][guard:-guard].view(shape)  # noqa: E731
    pg.vocab_ce_grad(h, W, t, view("loss", (N,)), view("gh", (N, d)), view("gw", (V, d)), ws[guard:-guard], lse=view("lse", (N,)))
    torch.cuda.synchronize()
    for b in bufs.values():
        assert (b[:guard] == 7.5).all() and (b[-guard:] == 7.5).all()
    assert (ws[:guard] == 0x5A).all() and (ws[-guard:] == 0x5A).all()
    check_grads(reference(h, W, t), view("gh", (N, d)), view("gw", (V, d)))


def test_no_rows(cuda):
    pg = _pg()
    W = torch.randn(10, 8, device=cuda)
    h, t, f = torch.empty(0, 8, device=cuda), torch.empty(0, dtype=torch.int32, device=cuda), torch.empty(0, device=cuda)
    gw = torch.full((10, 8), 3.0, device=cuda)
    pg.vocab_ce(h, W, t, f, None)
    pg.vocab_ce_grad(h, W, t, f, h.clone(), gw, None, accumulate=True)
    assert (gw == 3).all()
    pg.vocab_ce_grad(h, W, t, f, h.clone(), gw, None)
    assert (gw == 0).all()
    pg.vocab_distill_grad(h, W, torch.empty(0, 3, dtype=torch.int32, device=cuda), torch.empty(0, 3, device=cuda), f, None, gw, None)


@pytest.mark.parametrize("gwd", [F32, BF16])
@pytest.mark.parametrize("N", NS)
def test_accumulate(cuda, N, gwd):
    h, W, t = make(N, N, 700, 80, BF16, BF16, cuda)
    old = torch.randn(700, 80, generator=torch.Generator().manual_seed(N)).to(gwd).to(cuda)
    r = reference(h, W, t)
    gw = old.clone()
    _, _, _, dW = run_ce(h, W, t, None, gwd, accumulate=gw)
    assert dW is gw
    check_grads(r, None, gw, old)


@pytest.mark.parametrize("N", NS)
def test_equal_inputs_give_equal_bits(cuda, N):
    h, W, t, ids, u = make(N, N, 3000, 200, BF16, BF16, cuda, K=30)
    a = [run_ce(h, W, t, BF16, F32) + run_distill(h, W, ids, u, F32, BF16) for _ in range(3)]
    for b in a[1:]:
        for x, y in zip(a[0], b):
            assert torch.equal(x, y)


def test_one_workspace_for_calls_in_turn(cuda):
    # no synchronisation between them; larger and smaller calls leave their remains to each other
    pg = _pg()
    cases = []
    for i, (N, V, d, K) in enumerate([(300, 900, 72, 5), (40, 2000, 64, 9), (700, 300, 40, 256), (1, 50, 8, 1), (300, 900, 72, 5)]):
        cases.append(make(i, N, V, d, BF16, BF16, cuda, K=K))
    size = max(pg.vocab_distill_grad_workspace_size(h.shape[0], W.shape[0], h.shape[1], ids.shape[1], 1, 1, 1, 0)
               for h, W, _, ids, _ in cases)
    size = max(size, *(pg.vocab_ce_grad_workspace_size(h.shape[0], W.shape[0], h.shape[1], 1, 1, 1, 0) for h, W, *_ in cases))
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=cuda)
    outs = []
    for _ in range(3):
        for h, W, t, ids, u in cases:
            o = [torch.empty(h.shape[0], device=cuda), torch.empty_like(h), torch.empty(W.shape, device=cuda)]
            pg.vocab_ce_grad(h, W, t, o[0], o[1], o[2], ws)
            p = [torch.empty(h.shape[0], device=cuda), torch.empty_like(h), torch.empty(W.shape, device=cuda)]
            pg.vocab_distill_grad(h, W, ids, u, p[0], p[1], p[2], ws)
            outs.append(o + p)
    for i, o in enumerate(outs):
        h, W, t, ids, u = cases[i % len(cases)]
        if i < len(cases):
            check_grads(reference(h, W, t), o[1], o[2])
            check_grads(reference(h, W, ids=ids, u=u), o[4], o[5])
        else:
            assert all(torch.equal(x, y) for x, y in zip(o, outs[i % len(cases)])), i


def test_two_streams_at_once(cuda):
    pg = _pg()
    cases = [make(50 + i, N, 5000, 256, BF16, BF16, cuda) for i, N in enumerate((512, 100))]
    want = [run_ce(h, W, t, BF16, BF16) for h, W, t in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = []
    for rep in range(10):
        for (h, W, t), s in zip(cases, streams):
            with torch.cuda.stream(s):
                o = [torch.empty(h.shape[0], device=cuda), torch.empty_like(h), torch.empty_like(W)]
                ws = torch.empty(pg.vocab_ce_grad_workspace_size(h.shape[0], 5000, 256, 1, 1, 1, 1), dtype=torch.uint8, device=cuda)
                if rep % 2:
                    pg.vocab_ce_grad(h, W, t, o[0], o[1], o[2], ws)
                else:
                    pg.vocab_ce_grad(h, W, t, o[0], o[1], o[2], ws, stream=s)
                outs.append((o, ws))
    torch.cuda.synchronize()
    assert pg.device_error() == 0
    for i, (o, _) in enumerate(outs):
        w = want[i % 2]
        assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[2]) and torch.equal(o[2], w[3]), i


@pytest.mark.parametrize("N", NS)
def test_captured_and_replayed(cuda, N):
    # a step of loss and gradients in a graph, replayed on other inputs, between eager calls that use the same workspace
    pg = _pg()
    sets = [make(70 + i, N, 900, 72, BF16, BF16, cuda, K=6) for i in range(3)]
    h, W, t, ids, u = [x.clone() for x in sets[0]]
    size = max(pg.vocab_ce_grad_workspace_size(N, 900, 72, 1, 1, 1, 0), pg.vocab_distill_grad_workspace_size(N, 900, 72, 6, 1, 1, 1, 0))
    ws = torch.empty(size, dtype=torch.uint8, device=cuda)
    o = [torch.empty(N, device=cuda), torch.empty_like(h), torch.empty(900, 72, device=cuda),
         torch.empty(N, device=cuda), torch.empty_like(h), torch.empty(900, 72, device=cuda)]

    def step():
        pg.vocab_ce_grad(h, W, t, o[0], o[1], o[2], ws)
        pg.vocab_distill_grad(h, W, ids, u, o[3], o[4], o[5], ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    want = {}
    for rep in range(2):
        for i, s in enumerate(sets):
            for a, b in zip((h, W, t, ids, u), s):
                a.copy_(b)
            for x in o:
                x.fill_(float("nan"))
            graph.replay()
            got = [x.clone() for x in o]
            step()
            assert all(torch.equal(x, y) for x, y in zip(o, got)), (rep, i)
            if i in want:
                assert all(torch.equal(x, y) for x, y in zip(want[i], got))
            want[i] = got
    check_grads(reference(*sets[2][:3]), want[2][1], want[2][2])


def test_launches_are_counted(cuda):
    pg = _pg()
    h, W, t = make(1, 300, 700, 80, BF16, BF16, cuda)
    before = pg.launch_count()
    run_ce(h, W, t)
    assert pg.launch_count() == before + 3   # targets, logits, rows
    run_ce(h, W, t, BF16, BF16)
    assert before + 7 <= pg.launch_count() <= before + 8


@pytest.mark.parametrize("N", [3, 140])
def test_offsets_past_32_bits(cuda, N):
    # a table of 2.2e9 values
    V, d = 1_700_003, 1296
    pg = _pg()
    gen = torch.Generator(device=cuda).manual_seed(5)
    W = torch.empty(V, d, dtype=BF16, device=cuda)
    for lo in range(0, V, 100_000):
        W[lo:lo + 100_000] = torch.randn(W[lo:lo + 100_000].shape, generator=gen, device=cuda) / 36
    h = torch.randn(N, d, generator=gen, device=cuda).to(BF16)
    t = torch.randint(V - 5000, V, (N,), generator=gen, device=cuda).int()
    t[0] = V - 1
    gw = torch.full((V, d), float("nan"), dtype=BF16, device=cuda)
    loss, lse = torch.empty(N, device=cuda), torch.empty(N, device=cuda)
    gh = torch.empty(N, d, dtype=BF16, device=cuda)
    ws = torch.empty(pg.vocab_ce_grad_workspace_size(N, V, d, 1, 1, 1, 1), dtype=torch.uint8, device=cuda)
    pg.vocab_ce_grad(h, W, t, loss, gh, gw, ws, lse=lse)
    assert pg.device_error() == 0
    z = torch.cat([h.double() @ W[lo:lo + 200_000].double().T for lo in range(0, V, 200_000)], 1)
    want = torch.logsumexp(z, 1)
    assert (lse.double() - want).abs().max() <= 1e-4
    p = torch.softmax(z, 1)
    p[torch.arange(N), t.long()] -= 1
    for lo in (0, 1_000_000, V - 6000):  # the rows at both ends and between
        ref = p[:, lo:lo + 6000].T @ h.double()
        tol = (2 * half_step(BF16) + 1e-3) * (p[:, lo:lo + 6000].abs().T @ h.double().abs()) + half_step(BF16) * ref.abs()
        assert ((gw[lo:lo + 6000].double() - ref).abs() <= tol + 1e-12).all()
    dh = sum(p[:, lo:lo + 200_000] @ W[lo:lo + 200_000].double() for lo in range(0, V, 200_000))
    assert float((gh.double() - dh).norm() / dh.norm()) <= 2.0 ** -7
    assert not gw.isnan().any()


def test_a_workspace_serves_calls_of_fewer_rows(cuda):
    pg = _pg()
    h, W, t, ids, u = make(90, 1500, 2000, 264, BF16, BF16, cuda, K=20)
    size = pg.vocab_distill_grad_workspace_size(1500, 2000, 264, 20, 1, 1, 1, 0)
    ws = torch.full((size + 512,), 0x5A, dtype=torch.uint8, device=cuda)
    for N in (1500, 1, 31, 64, 128, 129, 255, 257, 400, 513, 1024, 1499):
        o = [torch.empty(N, device=cuda), torch.empty(N, 264, dtype=BF16, device=cuda), torch.empty(2000, 264, device=cuda)]
        pg.vocab_distill_grad(h[:N], W, ids[:N], u[:N], *o, ws[:size])
        check_grads(reference(h[:N], W, ids=ids[:N], u=u[:N]), o[1], o[2])
        assert (ws[size:] == 0x5A).all()
    assert pg.device_error() == 0


@pytest.mark.parametrize("N", [5, 150])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_the_widest_rows(cuda, N, dt):
    h, W, t = make(N, N, 300, 16384, dt, dt, cuda)
    r = reference(h, W, t)
    loss, lse, dh, dW = run_ce(h, W, t, dt, dt)
    check_values(r, loss, lse)
    check_grads(r, dh, dW)


def test_the_largest_vocabulary(cuda):
    V, N, d = (1 << 24) - 1, 3, 8
    gen = torch.Generator(device=cuda).manual_seed(6)
    W = torch.randn(V, d, generator=gen, device=cuda).to(BF16)
    h = torch.randn(N, d, generator=gen, device=cuda).to(BF16)
    ids = torch.tensor([[V - 1, 0, V - 1, 12345678], [V, V - 2, -1, 5], [V - 1, V, -7, V + 1]], dtype=torch.int32, device=cuda)
    u = torch.tensor([[1.0, 2.0, 0.5, -1.0], [3.0, 0.0, 9.0, 0.5], [1.0, 5.0, 6.0, 7.0]], device=cuda)
    r = reference(h, W, ids=ids, u=u)
    loss, lse, dh, dW = run_distill(h, W, ids, u, BF16, BF16)
    check_values(r, loss, lse)
    check_grads(r, dh, dW)
    t = torch.tensor([V - 1, V, 0], dtype=torch.int32, device=cuda)
    loss, lse, _, _ = run_ce(h, W, t)
    check_values(reference(h, W, t, grads=False), loss, lse)


@pytest.mark.parametrize("N", NS)
def test_what_is_left_out(cuda, N):
    # no loss, no lse, one gradient or none; scales of zero; a workspace that starts on 16 bytes
    pg = _pg()
    h, W, t, ids, u = make(N, N, 700, 80, BF16, BF16, cuda, K=5)
    full = run_ce(h, W, t, BF16, BF16)
    for ghd, gwd in [(1, None), (None, 1), (None, None)]:
        size = pg.vocab_ce_grad_workspace_size(N, 700, 80, 1, 1, ghd, gwd)
        ws = torch.empty(size + 16, dtype=torch.uint8, device=cuda)[16:]
        gh = None if ghd is None else torch.empty_like(h)
        gw = None if gwd is None else torch.empty_like(W)
        pg.vocab_ce_grad(h, W, t, None, gh, gw, ws)
        assert gh is None or torch.equal(gh, full[2])
        assert gw is None or torch.equal(gw, full[3])
    loss, lse, dh, dW = run_ce(h, W, t, BF16, F32, scale=0.0)
    keep = (t >= 0) & (t < 700)
    assert ((lse - math.log(700)).abs() <= 1e-5)[keep].all() and (dh == 0).all() and (dW == 0).all()
    _, _, dh, dW = run_distill(h, W, ids, u, BF16, F32, grad_scale=0.0)
    assert (dh == 0).all() and (dW == 0).all()
    with pytest.raises(ValueError, match="contiguous"):
        pg.vocab_ce(h[:, ::2], W[:, ::2], t, torch.empty(N, device=cuda), None)
    with pytest.raises(pg.PgError):
        pg.vocab_ce(h, W, t, torch.empty(N, device=cuda), torch.empty(100, dtype=torch.uint8, device=cuda))


# Up to 8 rows of an fp32 table have kernels of their own; d = 100 and 33: four values at a time, and one
@pytest.mark.parametrize("d", [100, 33])
@pytest.mark.parametrize("hdt", [F32, BF16])
def test_few_rows_of_an_fp32_table_in_every_way(cuda, d, hdt):
    pg = _pg()
    N, V = 7, 3001
    h, W, t = make(d, N, V, d, hdt, F32, cuda)
    t[:2] = torch.tensor([-1, V], device=cuda)
    t[2:4] = torch.tensor([0, V - 1], device=cuda)
    weight = torch.tensor([1.0, 2.0, 0.5, 1.0, 0.0, 3.0, 1.0], device=cuda)
    r = reference(h, W, t, weight=weight, z_loss=1e-3)
    first = run_ce(h, W, t, hdt, F32, weight=weight, z_loss=1e-3)
    check_values(r, first[0], first[1], 1e-3)
    check_grads(r, first[2], first[3])
    for fill in (float("nan"), float("inf"), torch.finfo(hdt).max):  # padded rows hold anything
        h2 = h.clone()
        h2[:2] = fill
        assert all(torch.equal(a, b) for a, b in zip(first, run_ce(h2, W, t, hdt, F32, weight=weight, z_loss=1e-3)))
    h2 = h.clone()
    h2[4] = float("nan")  # a row of weight zero has no gradient, whatever its loss
    second = run_ce(h2, W, t, hdt, F32, weight=weight, z_loss=1e-3)
    assert torch.equal(first[2], second[2]) and torch.equal(first[3], second[3])
    # guards around outputs and workspace; another stream, then a graph replayed on other inputs
    size = pg.vocab_ce_grad_workspace_size(N, V, d, pg.dtype_code(hdt), 0, 0, 0)
    guard = 512
    bufs = [torch.full((n + 2 * guard,), 7.5, device=cuda) for n in (N, N * d, V * d)]
    ws = torch.full((size + 2 * guard,), 0x5A, dtype=torch.uint8, device=cuda)
    loss, gh, gw = (b[guard:-guard].view(s) for b, s in zip(bufs, [(N,), (N, d), (V, d)]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pg.vocab_ce_grad(h, W, t, loss, gh, gw, ws[guard:-guard])
    torch.cuda.current_stream().wait_stream(side)
    check_grads(reference(h, W, t), gh, gw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pg.vocab_ce_grad(h, W, t, loss, gh, gw, ws[guard:-guard])
    for seed in (5, 6):
        for a, b in zip((h, W, t), make(seed, N, V, d, hdt, F32, cuda)):
            a.copy_(b)
        graph.replay()
        got = [x.clone() for x in (loss, gh, gw)]
        pg.vocab_ce_grad(h, W, t, loss, gh, gw, ws[guard:-guard])
        assert all(torch.equal(a, b) for a, b in zip(got, (loss, gh, gw)))
        check_grads(reference(h, W, t), gh, gw)
    torch.cuda.synchronize()
    assert pg.device_error() == 0
    for b in bufs:
        assert (b[:guard] == 7.5).all() and (b[-guard:] == 7.5).all()
    assert (ws[:guard] == 0x5A).all() and (ws[-guard:] == 0x5A).all()


@pytest.mark.parametrize("V,d", [(1100, 16384), (1 << 22, 8)])
def test_few_rows_of_the_widest_and_longest_fp32_tables(cuda, V, d):
    h, W, t = make(V, 8, V, d, F32, F32, cuda)
    r = reference(h, W, t)
    loss, lse, dh, dW = run_ce(h, W, t, F32, F32)
    check_values(r, loss, lse)
    check_grads(r, dh, dW)
