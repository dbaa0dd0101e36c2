"""The vocabulary losses without a GPU: sizes, refusals and the order of their host checks. Every refusal here is answered
before any CUDA work, so made-up (never touched) addresses stand for device pointers."""
import ctypes
import math

import pytest
import torch

NULL, SHAPE, DTYPE, ALIGN, UNSUPPORTED, WORKSPACE, DEVICE = 1, 2, 3, 5, 6, 8, 10
P = ctypes.c_void_p(1 << 20)   # aligned to everything
ODD = ctypes.c_void_p((1 << 20) + 1)
TWO = ctypes.c_void_p((1 << 20) + 2)
EIGHT = ctypes.c_void_p((1 << 20) + 8)
BIG = 1 << 50                  # a workspace size that is always enough

needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only where nothing can launch")


@pytest.fixture(scope="module")
def pg():
    from hashed_head_gram_gb300.build import build
    build()
    from hashed_head_gram_gb300 import pg as mod
    return mod


def ce(L, h=P, hdt=1, N=4, W=P, wdt=1, V=10, d=8, t=P, scale=1.0, zl=0.0, loss=P, lse=None, ws=P, wsb=BIG, err=None):
    return L.pg_vocab_ce(h, hdt, N, W, wdt, V, d, t, scale, zl, loss, lse, ws, wsb, err, None)


def ce_grad(L, h=P, hdt=1, N=4, W=P, wdt=1, V=10, d=8, t=P, scale=1.0, zl=0.0, rw=None, gs=1.0, loss=P, lse=None, gh=P, ghd=1,
            gw=P, gwd=1, acc=0, ws=P, wsb=BIG, err=None):
    return L.pg_vocab_ce_grad(h, hdt, N, W, wdt, V, d, t, scale, zl, rw, gs, loss, lse, gh, ghd, gw, gwd, acc, ws, wsb, err, None)


def distill(L, h=P, hdt=1, N=4, W=P, wdt=1, V=10, d=8, ids=P, u=P, udt=0, K=3, scale=1.0, T=1.0, loss=P, lse=None, ws=P, wsb=BIG,
            err=None):
    return L.pg_vocab_distill(h, hdt, N, W, wdt, V, d, ids, u, udt, K, scale, T, loss, lse, ws, wsb, err, None)


def distill_grad(L, h=P, hdt=1, N=4, W=P, wdt=1, V=10, d=8, ids=P, u=P, udt=0, K=3, scale=1.0, T=1.0, rw=None, gs=1.0, loss=P,
                 lse=None, gh=P, ghd=1, gw=P, gwd=1, acc=0, ws=P, wsb=BIG, err=None):
    return L.pg_vocab_distill_grad(h, hdt, N, W, wdt, V, d, ids, u, udt, K, scale, T, rw, gs, loss, lse, gh, ghd, gw, gwd, acc, ws,
                                   wsb, err, None)


COMMON = [
    (dict(N=-1), SHAPE), (dict(N=1 << 31), SHAPE), (dict(V=0), SHAPE), (dict(V=1 << 24), SHAPE), (dict(d=0), SHAPE),
    (dict(d=16385), SHAPE), (dict(hdt=2), DTYPE), (dict(wdt=-1), DTYPE), (dict(h=None), NULL), (dict(W=None), NULL),
    (dict(h=EIGHT), ALIGN), (dict(W=EIGHT), ALIGN),                       # read in place: 16 bytes
    (dict(h=TWO, d=7), DEVICE), (dict(W=TWO, d=7), DEVICE),               # copied first: an element's
    (dict(h=TWO, hdt=0), ALIGN), (dict(h=EIGHT, hdt=0), DEVICE), (dict(W=TWO, wdt=0), ALIGN), (dict(loss=TWO), ALIGN), (dict(lse=TWO), ALIGN),
    (dict(ws=EIGHT), ALIGN), (dict(ws=None), WORKSPACE), (dict(wsb=1000), WORKSPACE), (dict(err=TWO), ALIGN),
    (dict(scale=math.nan), UNSUPPORTED), (dict(scale=math.inf), UNSUPPORTED), (dict(), DEVICE)]
CE = [(dict(t=None), NULL), (dict(t=TWO), ALIGN), (dict(zl=math.inf), UNSUPPORTED), (dict(zl=math.nan), UNSUPPORTED)]
LIST = [(dict(ids=None), NULL), (dict(u=None), NULL), (dict(ids=TWO), ALIGN), (dict(u=TWO), ALIGN), (dict(u=TWO, udt=1), DEVICE),
        (dict(u=ODD, udt=1), ALIGN), (dict(udt=2), DTYPE), (dict(udt=-1), DTYPE), (dict(K=0), SHAPE), (dict(K=257), SHAPE),
        (dict(K=256), DEVICE), (dict(T=0.0), UNSUPPORTED), (dict(T=-1.0), UNSUPPORTED), (dict(T=math.nan), UNSUPPORTED),
        (dict(T=math.inf), UNSUPPORTED), (dict(T=1e-45), UNSUPPORTED), (dict(T=1e-38, scale=100.0), UNSUPPORTED)]
VALUES = [(dict(N=0, h=None, W=None, loss=None, ws=None, wsb=0), 0), (dict(loss=None), NULL)]
GRADS = [(dict(ghd=2), DTYPE), (dict(gwd=-2), DTYPE), (dict(gh=None), NULL), (dict(gw=None), NULL), (dict(gh=ODD), ALIGN), (dict(gw=ODD), ALIGN),
         (dict(gh=TWO), DEVICE), (dict(gw=TWO), DEVICE), (dict(gh=TWO, ghd=0), ALIGN), (dict(gw=TWO, gwd=0), ALIGN),
         (dict(gh=None, ghd=-1), DEVICE), (dict(gw=None, gwd=-1), DEVICE), (dict(gh=None, ghd=-1, gw=None, gwd=-1), DEVICE),
         (dict(loss=None), DEVICE), (dict(rw=TWO), ALIGN), (dict(gs=math.nan), UNSUPPORTED), (dict(gs=math.inf), UNSUPPORTED),
         (dict(N=0, gwd=-1, gw=None), 0), (dict(N=0, acc=1, gw=None), 0), (dict(N=0, gw=None), NULL), (dict(N=0, h=None, W=None, ws=None), DEVICE)]


@needs_no_gpu
@pytest.mark.parametrize("call,cases", [(ce, COMMON + CE + VALUES), (distill, COMMON + LIST + VALUES), (ce_grad, COMMON + CE + GRADS),
                                        (distill_grad, COMMON + LIST + GRADS)], ids=["ce", "distill", "ce_grad", "distill_grad"])
def test_refusals(pg, call, cases):
    for kw, want in cases:
        assert call(pg.lib(), **kw) == want, kw


def test_workspace_queries(pg):
    L = pg.lib()
    b = ctypes.c_size_t()
    assert L.pg_vocab_ce_workspace_size(4, 10, 8, 1, 1, None) == NULL
    assert L.pg_vocab_ce_grad_workspace_size(4, 10, 8, 1, 1, 1, 1, None) == NULL
    assert L.pg_vocab_distill_workspace_size(4, 10, 8, 257, 1, 1, ctypes.byref(b)) == SHAPE
    assert L.pg_vocab_distill_grad_workspace_size(4, 10, 8, 3, 1, 1, 3, 1, ctypes.byref(b)) == DTYPE
    assert L.pg_vocab_ce_workspace_size(4, 10, 8, 2, 1, ctypes.byref(b)) == DTYPE
    assert pg.vocab_ce_workspace_size(0, 10, 8, 1, 1) == 0
    assert pg.vocab_ce_grad_workspace_size(0, 10, 8, 1, 1, 1, None) == 0
    # exp of the logits for a chunk of rows, 2 GiB at most, however many rows there are
    small = pg.vocab_ce_grad_workspace_size(4096, 50304, 768, 1, 1, 1, 1)
    assert 2 * 4096 * 50304 <= small <= 2 * 4096 * 50304 + (1 << 28)
    assert pg.vocab_ce_grad_workspace_size(4, 100, 8, 1, 1, 1, 1) <= 1 << 20
    for N in (65536, 1 << 24, (1 << 31) - 1):
        assert pg.vocab_ce_grad_workspace_size(N, 50304, 768, 1, 1, 1, 1) <= (2 << 30) + (1 << 30)
    # the forward call keeps sums and, of fp32 operands, their pieces; up to 8 rows take W as it is
    assert pg.vocab_ce_workspace_size(1 << 20, 50304, 768, 1, 1) <= 1 << 28
    assert pg.vocab_ce_workspace_size(64, 50304, 768, 1, 0) >= 6 * 50304 * 768
    assert pg.vocab_ce_workspace_size(8, 50304, 768, 1, 0) <= 1 << 24
    assert pg.vocab_ce_grad_workspace_size(8, 1024, 768, 1, 0, 1, 1) >= 6 * 1024 * 768
    assert pg.vocab_distill_workspace_size(4096, 50304, 768, 64, 1, 1) >= 12 * 4096 * 64
    # sizes at both ends
    for N, V, d in [(1, 1, 1), (1, (1 << 24) - 1, 1), (1, 1, 16384), ((1 << 31) - 1, 1, 1), ((1 << 31) - 1, (1 << 24) - 1, 16384)]:
        for dt in (0, 1):
            assert pg.vocab_ce_workspace_size(N, V, d, dt, dt) > 0
            assert pg.vocab_ce_grad_workspace_size(N, V, d, dt, dt, dt, dt) > 0
            assert pg.vocab_distill_grad_workspace_size(N, V, d, 256, dt, dt, None, dt) > 0


@pytest.mark.parametrize("V,d", [(1, 1), (10, 8), (300, 72), (1024, 256), (5000, 2560), (50304, 768), (128000, 33)])
def test_a_workspace_serves_fewer_rows(pg, V, d):
    rows = sorted({*range(1, 140), *(128 * k + r for k in range(1, 90) for r in (-1, 0, 1)), *(2 ** k + r for k in range(13, 31) for r in (-1, 0, 1)),
                   *(int(1.13 ** k) for k in range(60, 175))})
    for hd, wd, ghd, gwd in [(1, 1, 1, 1), (0, 0, 0, 0), (1, 1, None, 0), (1, 0, 0, None), (1, 1, 1, 0)]:
        last = [0] * 4
        for N in rows:
            now = [pg.vocab_ce_workspace_size(N, V, d, hd, wd), pg.vocab_ce_grad_workspace_size(N, V, d, hd, wd, ghd, gwd),
                   pg.vocab_distill_workspace_size(N, V, d, 30, hd, wd), pg.vocab_distill_grad_workspace_size(N, V, d, 30, hd, wd, ghd, gwd)]
            assert all(a >= b for a, b in zip(now, last)), (N, now, last)
            last = now


def test_binding_checks_sizes_and_types(pg):
    t = torch.zeros(4, dtype=torch.int32)
    h, W, f = torch.zeros(4, 8), torch.zeros(10, 8), torch.zeros(4)
    ids, u = torch.zeros(4, 3, dtype=torch.int32), torch.zeros(4, 3)
    for bad in [dict(h=torch.zeros(4, 7)), dict(W=torch.zeros(8)), dict(targets=t.long()), dict(targets=t[:3]), dict(loss=f[:3]),
                dict(loss=f.double()), dict(lse=torch.zeros(4, 1)), dict(err_index=f), dict(h=h.half()), dict(W=W.double())]:
        with pytest.raises(ValueError):
            pg.vocab_ce(**{**dict(h=h, W=W, targets=t, loss=f, workspace=None), **bad})
    good = dict(h=h, W=W, targets=t, loss=None, grad_h=h, grad_W=W, workspace=None)
    for bad in [dict(grad_h=W), dict(grad_W=h), dict(grad_h=h.half()), dict(row_weight=t), dict(row_weight=torch.zeros(5))]:
        with pytest.raises(ValueError):
            pg.vocab_ce_grad(**{**good, **bad})
    good = dict(h=h, W=W, teacher_ids=ids, teacher_logits=u, loss=f, workspace=None)
    for bad in [dict(teacher_ids=ids.long()), dict(teacher_ids=ids[:3]), dict(teacher_ids=t), dict(teacher_logits=u[:, :2]),
                dict(teacher_logits=u.half())]:
        with pytest.raises(ValueError):
            pg.vocab_distill(**{**good, **bad})
        with pytest.raises(ValueError):
            pg.vocab_distill_grad(grad_h=None, grad_W=None, **{**good, **bad})
    # well-formed, but not on a GPU
    for call in (lambda: pg.vocab_ce(h, W, t, f, None), lambda: pg.vocab_ce_grad(h, W, t, f, h, None, None),
                 lambda: pg.vocab_distill(h, W, ids, u, f, None), lambda: pg.vocab_distill_grad(h, W, ids, u, f, None, W, None)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_star_import_has_the_losses(pg):
    names = {}
    exec("from hashed_head_gram_gb300.pg import *", names)
    for call in ("vocab_ce", "vocab_ce_grad", "vocab_distill", "vocab_distill_grad"):
        assert names[call] is getattr(pg, call)
        assert names[call + "_workspace_size"] is getattr(pg, call + "_workspace_size")
