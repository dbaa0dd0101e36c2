"""The training calls without a GPU: sizes, refusals and the order of their host checks. Every
refusal here is answered before any CUDA work, so made-up (never touched) addresses stand for
device pointers."""
import ctypes
import dataclasses

import pytest
import torch

from hashed_head_gram_gb300 import workloads as W

NULL, SHAPE, DTYPE, ALIGN, UNSUPPORTED, VERSION, WORKSPACE, DEVICE = 1, 2, 3, 5, 6, 7, 8, 10
P = ctypes.c_void_p(1 << 20)   # aligned to everything
ODD = ctypes.c_void_p((1 << 20) + 1)
TWO = ctypes.c_void_p((1 << 20) + 2)
BIG = 1 << 40                  # a workspace size that is always enough

needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only where nothing can launch")


@pytest.fixture(scope="module")
def pg():
    from hashed_head_gram_gb300.build import build
    build()
    from hashed_head_gram_gb300 import pg as mod
    return mod


def embed(L, tokens=P, N=4, vocab=10, cmap=None, table=P, tdt=0, rows=10, d=8, out=P, odt=0, err=None):
    return L.pg_embed(tokens, N, vocab, cmap, table, tdt, rows, d, 1.0, out, odt, err, None)


def embed_grad(L, tokens=P, N=4, vocab=10, cmap=None, g=P, gdt=0, rows=10, d=8, acc=0, out=P, odt=0, ws=P, wsb=BIG,
               err=None):
    return L.pg_embed_grad(tokens, N, vocab, cmap, g, gdt, rows, d, 1.0, acc, out, odt, ws, wsb, err, None)


def lookup_grad(L, desc, tokens=P, B=2, T=3, cmap=None, g=P, gdt=0, rows=P, out=P, odt=0, count=P, ws=P, wsb=BIG,
                err=None):
    return L.pg_lookup_grad(ctypes.byref(desc), tokens, B, T, cmap, g, gdt, rows, out, odt, count, ws, wsb, err, None)


def ortho(L, G=P, dt=1, batch=1, m=8, n=8, steps=5, out=P, ws=P, wsb=BIG):
    return L.pg_orthogonalize(G, dt, batch, m, n, steps, 3.0, -4.0, 2.0, 1e-7, 1.0, out, ws, wsb, None)


@needs_no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(N=-1), SHAPE), (dict(N=1 << 31), SHAPE), (dict(vocab=0), SHAPE), (dict(rows=0), SHAPE),
    (dict(rows=1 << 31), SHAPE), (dict(d=0), SHAPE), (dict(d=(1 << 20) + 1), SHAPE), (dict(tdt=2), DTYPE),
    (dict(odt=2), DTYPE), (dict(odt=-1), DTYPE), (dict(N=0, tokens=None, table=None, out=None), 0),
    (dict(tokens=None), NULL), (dict(table=None), NULL), (dict(out=None), NULL), (dict(tokens=TWO), ALIGN),
    (dict(cmap=TWO), ALIGN), (dict(table=TWO), ALIGN), (dict(table=TWO, tdt=1), DEVICE), (dict(out=ODD, odt=1), ALIGN),
    (dict(err=TWO), ALIGN), (dict(), DEVICE)])
def test_embed_refusals(pg, kw, want):
    assert embed(pg.lib(), **kw) == want


@needs_no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(N=-1), SHAPE), (dict(N=1 << 31), SHAPE), (dict(vocab=0), SHAPE), (dict(rows=0), SHAPE), (dict(d=0), SHAPE),
    (dict(gdt=2), DTYPE), (dict(odt=3), DTYPE), (dict(tokens=None), NULL), (dict(g=None), NULL), (dict(out=None), NULL),
    (dict(N=0, out=None), NULL), (dict(g=TWO), ALIGN), (dict(out=TWO), ALIGN), (dict(ws=ctypes.c_void_p(8)), ALIGN),
    (dict(wsb=16), WORKSPACE), (dict(ws=None), WORKSPACE), (dict(err=ODD), ALIGN), (dict(), DEVICE),
    (dict(N=0, tokens=None, g=None, ws=None, wsb=0), DEVICE)])
def test_embed_grad_refusals(pg, kw, want):
    assert embed_grad(pg.lib(), **kw) == want


@needs_no_gpu
def test_lookup_grad_refusals(pg):
    L = pg.lib()
    spec = W.make_workload(2).tables[0]
    d = pg.table_desc(spec, 50304)
    for kw, want in [(dict(B=-1), SHAPE), (dict(T=-1), SHAPE), (dict(B=1 << 16, T=1 << 15), SHAPE),
                     (dict(B=1 << 14, T=1 << 13), SHAPE),  # 2^27 tokens, 2^31 reads
                     (dict(gdt=2), DTYPE), (dict(odt=2), DTYPE), (dict(tokens=None), NULL), (dict(g=None), NULL),
                     (dict(rows=None), NULL), (dict(out=None), NULL), (dict(count=None), NULL),
                     (dict(B=0, count=None), NULL), (dict(count=TWO), ALIGN), (dict(rows=TWO), ALIGN),
                     (dict(g=TWO), ALIGN), (dict(out=TWO), ALIGN), (dict(wsb=100), WORKSPACE), (dict(ws=None), WORKSPACE),
                     (dict(ws=TWO), ALIGN), (dict(), DEVICE)]:
        assert lookup_grad(L, d, **kw) == want, kw
    bad = pg.table_desc(spec, 50304)
    bad.abi_version = 3
    assert lookup_grad(L, bad) == VERSION
    many = pg.table_desc(dataclasses.replace(spec, K=16, orders=[1, 2, 3], pages=[5, 5, 5]), 50304)
    assert lookup_grad(L, many) == UNSUPPORTED          # 48 heads a token
    toy = pg.table_desc(W.TableSpec("toy", W.MODE_FLAT, K=1, S=1, r=8, row_dtype=0, orders=[2], rows=[[7]],
                                    hash_kind=W.HASH_TOY), 100)
    assert lookup_grad(L, toy) == UNSUPPORTED


@needs_no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(batch=-1), SHAPE), (dict(batch=4097), SHAPE), (dict(m=0), SHAPE), (dict(n=0), SHAPE), (dict(m=16385), SHAPE),
    (dict(steps=0), SHAPE), (dict(steps=33), SHAPE), (dict(dt=2), DTYPE), (dict(batch=0, G=None, out=None, ws=None), 0),
    (dict(G=None), NULL), (dict(out=None), NULL), (dict(G=TWO, dt=0), ALIGN), (dict(out=ODD), ALIGN), (dict(ws=TWO), ALIGN),
    (dict(wsb=8), WORKSPACE), (dict(ws=None), WORKSPACE), (dict(), DEVICE)])
def test_orthogonalize_refusals(pg, kw, want):
    assert ortho(pg.lib(), **kw) == want


def test_workspace_queries(pg):
    L = pg.lib()
    b = ctypes.c_size_t()
    assert L.pg_embed_grad_workspace_size(4, 10, 8, None) == NULL
    assert L.pg_embed_grad_workspace_size(-1, 10, 8, ctypes.byref(b)) == SHAPE
    assert pg.embed_grad_workspace_size(0, 10, 8) == 0
    assert pg.embed_grad_workspace_size(65536, 50304, 768) >= 16 * 65536   # keys and references, twice
    d = pg.table_desc(W.make_workload(5).tables[0], 128000)
    assert L.pg_lookup_grad_workspace_size(ctypes.byref(d), 4, None) == NULL
    assert L.pg_lookup_grad_workspace_size(ctypes.byref(d), 1 << 27, ctypes.byref(b)) == SHAPE
    assert pg.lookup_grad_workspace_size(d, 0) == 0
    assert pg.lookup_grad_workspace_size(d, 32768) >= 24 * 32768 * 16
    assert L.pg_orthogonalize_workspace_size(1, 8, 8, None) == NULL
    assert pg.orthogonalize_workspace_size(0, 8, 8) == 0
    # X twice and two [p, p] matrices, fp16
    assert pg.orthogonalize_workspace_size(5, 2560, 1280) >= 2 * 5 * (2 * 2560 * 1280 + 2 * 1280 * 1280)


def test_binding_checks_sizes_and_types(pg):
    t = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        pg.embed(t.long(), torch.zeros(10, 8), torch.zeros(4, 8), 10)
    with pytest.raises(ValueError):
        pg.embed(t, torch.zeros(10, 8), torch.zeros(4, 9), 10)
    with pytest.raises(ValueError):
        pg.embed(t, torch.zeros(10, 8), torch.zeros(4, 8), 10, canon_map=torch.zeros(9, dtype=torch.int32))
    with pytest.raises(ValueError):
        pg.embed(t, torch.zeros(10, 8), torch.zeros(4, 8), 10)          # not on a GPU
    with pytest.raises(ValueError):
        pg.embed_grad(t, torch.zeros(3, 8), torch.zeros(10, 8), 10, None)
    with pytest.raises(ValueError):
        pg.embed_grad(t, torch.zeros(4, 8, dtype=torch.float16), torch.zeros(10, 8), 10, None)
    with pytest.raises(ValueError):
        pg.orthogonalize(torch.zeros(4, 8), torch.zeros(4, 8), t)       # out is not bf16
    with pytest.raises(ValueError):
        pg.orthogonalize(torch.zeros(4, 8), torch.zeros(8, 4, dtype=torch.bfloat16), t)
    spec = W.make_workload(1).tables[0]
    d = pg.table_desc(spec, 1024)
    tok = torch.zeros(1, 4, dtype=torch.int32)
    good = dict(grad_e=torch.zeros(4, 1024), rows_out=torch.zeros(64, dtype=torch.int32), grads_out=torch.zeros(64, 64),
                count_out=torch.zeros(1, dtype=torch.int32), workspace=None)
    for k, v in [("grad_e", torch.zeros(4, 1000)), ("rows_out", torch.zeros(63, dtype=torch.int32)),
                 ("grads_out", torch.zeros(64, 63)), ("count_out", torch.zeros(1))]:
        with pytest.raises(ValueError):
            pg.lookup_grad(d, tok, **{**good, k: v})
