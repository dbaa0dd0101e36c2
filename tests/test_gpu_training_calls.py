"""Training calls one after the other: the workspace and the outputs of a call are the next one's."""
import pytest
import torch

from tests.test_gpu_training import BF16, F32, SPECS, _pg, make_ids

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,shift", [(64, 0), (264, 0), (33, 1)])
def test_calls_in_turn_on_one_workspace(cuda, d, shift):
    # the parts of rows that cross tiles are new in every call; integers, so that sums are exact
    pg = _pg()
    gen = torch.Generator().manual_seed(d)
    N, rows = 20_011, 40
    ws = torch.empty(pg.embed_grad_workspace_size(N, rows, d), dtype=torch.uint8, device=cuda)
    toks = [make_ids(gen, N, rows, kind, cuda) for kind in ("skewed", "same", "skewed", "skewed")]
    grads = [torch.randint(-4, 5, (N, d), generator=gen).to(BF16).to(cuda) for _ in toks]
    outs = [torch.empty(rows * d + shift, device=cuda)[shift:].view(rows, d) for _ in range(12)]
    for i, out in enumerate(outs):  # no synchronisation between them
        pg.embed_grad(toks[i % 4], grads[i % 4], out, rows, ws)
    for i, out in enumerate(outs):
        want = torch.zeros(rows, d, device=cuda).index_add_(0, toks[i % 4].long(), grads[i % 4].float())
        assert torch.equal(out, want), i


def test_lookup_gradients_in_turn_on_one_workspace(cuda):
    pg = _pg()
    spec = SPECS["pagegram"]()
    desc = pg.table_desc(spec, 300)
    gen = torch.Generator().manual_seed(5)
    tokens = make_ids(gen, 8000, 300, "skewed", cuda).view(2, 4000)
    n = 8000 * 16
    ws = torch.empty(pg.lookup_grad_workspace_size(desc, 8000), dtype=torch.uint8, device=cuda)
    grads = [torch.randn(8000, 1024, generator=gen).to(cuda) for _ in range(3)]
    got = []
    for i in range(9):
        got.append((torch.empty(n, dtype=torch.int32, device=cuda), torch.empty(n, 64, dtype=F32, device=cuda),
                    torch.empty(1, dtype=torch.int32, device=cuda)))
        pg.lookup_grad(desc, tokens, grads[i % 3], *got[-1], ws)
    for i in range(3, 9):  # equal inputs, equal bits
        for x, y in zip(got[i], got[i % 3]):
            assert torch.equal(x, y), i
    assert not torch.equal(got[0][1], got[1][1])
