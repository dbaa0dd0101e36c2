"""The losses with the calls they are used with: a memory under a tied embedding, as examples/train_memory.py trains it. The
embedding, lookup, projection, loss, its gradients, the embedding's and the table's gradients and the update run one after the
other on one workspace; the tied table's gradient is held against the formulas in 64 bits, and a step against its replay."""
import math

import pytest
import torch

from hashed_head_gram_gb300 import workloads as W
from tests.test_gpu_vocab import check_grads, check_values, reference

pytestmark = pytest.mark.gpu


def small(cuda, K=0, B=4, L=100, vocab=700, d=256):
    from examples.train_memory import Memory, TokenTrainer
    spec = W.TableSpec("memory", W.MODE_PAGEGRAM, K=8, S=4, r=64, row_dtype=W.DT_BF16, pages=[61, 59], hash_seed=7)
    gen = torch.Generator().manual_seed(B * L)
    tokens = torch.randint(0, vocab, (B, L), generator=gen, dtype=torch.int32).to(cuda)
    targets = torch.full_like(tokens, -1)
    targets[:, :-1] = tokens[:, 1:]
    trainer = TokenTrainer(Memory(spec, vocab, d, 3, cuda, std=1.0), B * L, K, logit_scale=2.0)
    ids = torch.randint(0, vocab, (B * L, max(K, 1)), generator=gen, dtype=torch.int32).to(cuda)
    u = torch.randn(B * L, max(K, 1), generator=gen).to(cuda)
    return trainer, tokens, targets, ((ids, u) if K else None)


@pytest.mark.parametrize("K", [0, 12])
@pytest.mark.parametrize("B,L", [(4, 100), (2, 11), (3, 700)])
def test_tied_gradients(cuda, B, L, K):
    from hashed_head_gram_gb300 import pg
    tr, tokens, targets, teacher = small(cuda, K, B, L)
    m, N = tr.model, B * L
    e, y, _ = tr.gradients(tokens, targets, teacher)
    assert pg.device_error() == 0
    kw = dict(target=targets.view(-1)) if K == 0 else dict(ids=teacher[0], u=teacher[1])
    r = reference(y, tr.E16, scale=tr.logit_scale, grad_scale=1.0 / N, **kw)
    lse = torch.where(r["keep"], r["lse"], 0.0)
    check_values(r, tr.loss, lse.float())
    # the two parts: the output table's, then the rows that the tokens read (adding them in fp32: 2^-22 of the magnitudes)
    inner = torch.zeros_like(r["dW"]).index_add_(0, tokens.view(-1).long(), m.scale * tr.dy.double())
    size = torch.zeros_like(r["dW"]).index_add_(0, tokens.view(-1).long(), m.scale * tr.dy.double().abs())
    counts = torch.bincount(tokens.view(-1).long(), minlength=m.vocab)[:, None]
    got = tr.dE.double() - inner
    slack = (counts + 4) * 2.0 ** -24 * size + 2.0 ** -23 * (inner.abs() + r["dW"].abs())
    tol = (r["off"] + 2.0 ** -21 * (r["dz"].abs() + r["off"])).T @ r["h"].abs() + (N + 16) * 2.0 ** -23 * (r["dz"].abs().T @ r["h"].abs())
    assert ((got - r["dW"]).abs() <= tol + slack).all()
    check_grads(r, tr.dy, None)


@pytest.mark.parametrize("K", [0, 12])
def test_a_step_replays(cuda, K):
    # the whole step in a graph: the same bits as the eager step from the same weights
    tr, tokens, targets, teacher = small(cuda, K)
    m = tr.model
    state = [m.E, m.T, m.W, tr.momentum]
    for _ in range(2):
        tr.step(tokens, targets, teacher)
    kept = [x.clone() for x in state]
    torch.cuda.synchronize()
    m.T16, m.W16 = m.T16.clone(), m.W16.clone()
    refresh16 = (m.T16, m.W16)

    def refresh():
        refresh16[0].copy_(m.T[:-1])
        refresh16[1].copy_(m.W)
    m.refresh = refresh
    m.T16, m.W16 = refresh16

    def restore():
        for x, k in zip(state, kept):
            x.copy_(k)
        refresh()

    restore()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want_loss = tr.step(tokens, targets, teacher).clone()
    torch.cuda.current_stream().wait_stream(side)
    want = [x.clone() for x in state]
    restore()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = tr.step(tokens, targets, teacher)
    for _ in range(2):
        restore()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, want_loss)
        # (the table's index_add_ adds rows that are distinct but for the spare one)
        for x, y in zip((m.E, m.T[:-1], m.W, tr.momentum), (want[0], want[1][:-1], want[2], want[3])):
            assert torch.equal(x, y)


@pytest.mark.parametrize("K", [0, 16])
def test_the_example_runs(cuda, K):
    from hashed_head_gram_gb300 import pg
    from examples.train_memory import train_tokens
    losses = train_tokens(steps=3, n_tokens=512, K=K)
    assert losses.shape == (3,) and bool(losses.isfinite().all()) and bool((losses > 0).all())
    assert pg.device_error() == 0


def test_perplexity_of_pieces(cuda):
    # scoring a sequence in pieces, down to single tokens, gives what scoring it at once gives
    from hashed_head_gram_gb300 import pg
    gen = torch.Generator().manual_seed(4)
    N, V, d = 300, 5000, 256
    h = torch.randn(N, d, generator=gen).bfloat16().to(cuda)
    Wt = (torch.randn(V, d, generator=gen) / 16).bfloat16().to(cuda)
    t = torch.randint(0, V, (N,), generator=gen, dtype=torch.int32).to(cuda)
    ws = torch.empty(pg.vocab_ce_workspace_size(N, V, d, 1, 1), dtype=torch.uint8, device=cuda)
    whole, loss = torch.empty(N, device=cuda), torch.empty(N, device=cuda)
    pg.vocab_ce(h, Wt, t, whole, ws)
    for cut in (1, 7, 33, 100, 299):
        pg.vocab_ce(h[:cut], Wt, t[:cut], loss[:cut], ws)
        pg.vocab_ce(h[cut:], Wt, t[cut:], loss[cut:], ws)
        # two fp32 sums of the same terms in other orders, each within E of check_values: d = 256, |z| < 8
        assert (loss - whole).abs().max() <= 4 * (d + 16) * 2.0 ** -23 * 16
    assert math.isfinite(float(whole.mean()))
