"""The training calls' host side (no GPU needed): coefficients, the binding's names and types."""
import ctypes
import math

import pytest
import torch

UNSUPPORTED, DEVICE = 6, 10
P = ctypes.c_void_p(1 << 20)   # never touched: every call here ends in its host checks

needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only where nothing can launch")


@pytest.fixture(scope="module")
def pg():
    from hashed_head_gram_gb300.build import build
    build()
    from hashed_head_gram_gb300 import pg as mod
    return mod


@needs_no_gpu
@pytest.mark.parametrize("coeffs,want", [
    ((3.4445, -4.7750, 2.0315), DEVICE), ((62.9, -1.0, 0.0), DEVICE), ((-62.9, 1.0, 0.0), DEVICE),
    ((3.0, -4.0, 2.0), DEVICE), ((63.0, 0.0, 0.0), UNSUPPORTED), ((-64.0, 0.0, 0.0), UNSUPPORTED),
    ((math.nan, 0.0, 0.0), UNSUPPORTED), ((1.0, math.inf, 0.0), UNSUPPORTED), ((1.0, 0.0, math.nan), UNSUPPORTED)])
def test_orthogonalize_coefficients(pg, coeffs, want):
    # a I is held in fp16 times 2^10
    got = pg.lib().pg_orthogonalize(P, 1, 1, 8, 8, 5, *coeffs, 1e-7, 1.0, P, P, 1 << 40, None)
    assert got == want


def test_star_import_has_the_training_calls(pg):
    names = {}
    exec("from hashed_head_gram_gb300.pg import *", names)
    for call in ("embed", "embed_grad", "lookup_grad", "orthogonalize"):
        assert names[call] is getattr(pg, call)
        if call != "embed":
            assert names[call + "_workspace_size"] is getattr(pg, call + "_workspace_size")
    assert names["selftest_training_waits"] is pg.selftest_training_waits


def test_ids_are_integers(pg):
    from hashed_head_gram_gb300 import workloads as W
    tok = torch.zeros(1, 4, dtype=torch.int32)
    table, out = torch.zeros(10, 8), torch.zeros(4, 8)
    for bad in (torch.zeros(10), torch.zeros(10, dtype=torch.int64)):
        with pytest.raises(ValueError, match="canon_map"):
            pg.embed(tok, table, out, 10, canon_map=bad)
        with pytest.raises(ValueError, match="canon_map"):
            pg.embed_grad(tok, out, table, 10, None, canon_map=bad)
    d = pg.table_desc(W.make_workload(1).tables[0], 1024)
    rest = (torch.zeros(64, 64), torch.zeros(1, dtype=torch.int32), None)
    with pytest.raises(ValueError, match="rows_out"):
        pg.lookup_grad(d, tok, torch.zeros(4, 1024), torch.zeros(64), *rest)
    for dtype in (torch.int32, torch.uint32):  # accepted: the next check is that they are on a GPU
        with pytest.raises(ValueError, match="CUDA"):
            pg.embed(tok, table, out, 10, canon_map=torch.zeros(10, dtype=dtype))
        with pytest.raises(ValueError, match="CUDA"):
            pg.lookup_grad(d, tok, torch.zeros(4, 1024), torch.zeros(64, dtype=dtype), *rest)
