"""The vocabulary losses where their rows come in chunks and their gradients in parts."""
import pytest
import torch

from tests.test_gpu_vocab import BF16, F32, _pg, check_grads, check_values, make, reference, run_ce, run_distill

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,V,d,K,ghd,gwd", [(6000, 70001, 40, 30, F32, BF16), (700_000, 64, 40, 256, BF16, BF16), (700_000, 64, 33, 200, None, F32)])
def test_lists_in_chunks(cuda, N, V, d, K, ghd, gwd):
    # 2 GiB hold 4800 rows of three pieces of 70,001 columns, or some 640,000 of 64 with lists of 256
    gen = torch.Generator(device=cuda).manual_seed(N + K)
    h, W, _ = make(3, 1, V, d, BF16, BF16, cuda)
    h = torch.randn(N, d, generator=gen, device=cuda).to(BF16)
    ids = torch.randint(-V // 8, V, (N, K), generator=gen, device=cuda, dtype=torch.int32)
    u = (torch.randn(N, K, generator=gen, device=cuda) * 2).to(BF16)
    r = reference(h, W, ids=ids, u=u, grad_scale=0.01)
    loss, lse, dh, dW = run_distill(h, W, ids, u, ghd, gwd, grad_scale=0.01)
    check_values(r, loss, lse)
    check_grads(r, dh, dW)


@pytest.mark.parametrize("hdt,gwd", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("N,V,d", [(20011, 300, 72), (9000, 1024, 256), (4097, 64, 33), (20011, 300, 33)])
def test_parts_are_added_to_what_is_there(cuda, N, V, d, hdt, gwd):
    # grad_W's few tiles are cut along the rows; joining the parts adds the old gradient (four columns at a time, and one)
    h, W, t = make(N + d, N, V, d, hdt, hdt, cuda)
    r = reference(h, W, t, grad_scale=1.0 / N)
    old = (torch.randn(V, d, generator=torch.Generator().manual_seed(N)) * 0.01).to(gwd).to(cuda)
    gw = old.clone()
    run_ce(h, W, t, BF16, gwd, grad_scale=1.0 / N, accumulate=gw)
    check_grads(r, None, gw, old)
    ids, u = t[:, None].contiguous(), torch.zeros(N, 1, device=cuda)
    pg = _pg()
    gw.copy_(old)
    loss = torch.empty(N, device=cuda)
    code = pg.dtype_code(hdt)
    ws = torch.empty(pg.vocab_distill_grad_workspace_size(N, V, d, 1, code, code, None, pg.dtype_code(gwd)), dtype=torch.uint8, device=cuda)
    pg.vocab_distill_grad(h, W, ids, u, loss, None, gw, ws, grad_scale=1.0 / N, accumulate=True)
    check_grads(r, None, gw, old)


def test_losses_take_no_device_memory(cuda):
    # all that the calls use is the caller's: outputs, gradients and workspace
    pg = _pg()
    cases = []
    for N, V, d, K, dt in [(8, 5000, 256, 20, BF16), (300, 5000, 256, 20, BF16), (5, 3000, 64, 7, F32), (200, 3000, 64, 7, F32)]:
        h, W, t, ids, u = make(N, N, V, d, dt, dt, cuda, K=K)
        code = pg.dtype_code(dt)
        size = max(pg.vocab_ce_grad_workspace_size(N, V, d, code, code, code, 0), pg.vocab_distill_grad_workspace_size(N, V, d, K, code, code, code, 0))
        cases.append((h, W, t, ids, u, torch.empty(N, device=cuda), torch.empty_like(h), torch.empty(V, d, device=cuda),
                      torch.empty(size, dtype=torch.uint8, device=cuda)))

    def calls():
        for h, W, t, ids, u, loss, gh, gw, ws in cases:
            pg.vocab_ce(h, W, t, loss, ws)
            pg.vocab_distill(h, W, ids, u, loss, ws)
            pg.vocab_ce_grad(h, W, t, loss, gh, gw, ws)
            pg.vocab_distill_grad(h, W, ids, u, loss, gh, gw, ws)

    calls()  # loads the device code
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    for _ in range(3):
        calls()
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == free
    assert pg.device_error() == 0


@pytest.mark.parametrize("N", [5, 300])
def test_a_list_whose_heaviest_token_is_out_of_reach(cuda, N):
    # its logit is -infinity in fp32: so is log q, and the loss infinite; what is pushed down and up is finite
    h, W, _, ids, u = make(N, N, 700, 80, F32, F32, cuda, K=4, pad=0.0)
    h[:, 0], W[:, 0] = 1e20, 0.0
    ids[:] = torch.tensor([7, 8, 9, 10], dtype=torch.int32, device=cuda)
    u[:] = torch.tensor([3.0, 0.0, 0.0, 0.0], device=cuda)
    W[7, 0] = -1e20
    loss, lse, _, dW = run_distill(h, W, ids, u, None, F32)
    assert (loss == float("inf")).all() and lse.isfinite().all()
    forward, _, _, _ = run_distill(h, W, ids, u)
    assert (forward == float("inf")).all()
    _, _, dh, _ = run_distill(h, W, ids, u, F32, None)
    assert dh[:, 1:].isfinite().all()
