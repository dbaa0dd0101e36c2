"""The bounded waits of the training calls give up and report instead of hanging, and what follows a
sort that did not finish writes nothing. The waits run out on counters that nothing completes, in
kernels without copies, tensor-core operations or TMEM; the calls then work as before."""
import time

import pytest
import torch

from tests.test_gpu_training import BF16, F32, check_embed_grad, gaussian, ortho_reference, rel, run_ortho

pytestmark = pytest.mark.gpu


def test_training_waits_give_up_and_report(cuda):
    from hashed_head_gram_gb300 import pg
    assert pg.device_error(clear=True) == 0
    scratch = torch.full((512,), 7, dtype=torch.int32, device=cuda)
    sums = torch.full((8,), 3.0, device=cuda)
    t0 = time.perf_counter()
    pg.selftest_training_waits(scratch, sums)
    code = pg.device_error(clear=True)                 # synchronizes
    took = time.perf_counter() - t0
    assert code == 131072 | 262144
    assert scratch[:3].tolist() == [1, 1, 1]
    assert 2.5 <= took <= 60.0                         # three waits of about 1 s each
    assert bool((sums == 3.0).all())                   # neither the sums nor the join wrote
    assert pg.device_error() == 0
    check_embed_grad(cuda, 3000, 40, 900, 700, "skewed", BF16, F32)
    G = gaussian(torch.Generator().manual_seed(1), 1, 130, 200, F32, cuda)
    assert rel(run_ortho(pg, G), ortho_reference(G, 5)) <= 2.0 ** -6


def test_training_selftest_refuses_bad_buffers(cuda):
    from hashed_head_gram_gb300 import pg
    scratch = torch.zeros(4096, dtype=torch.uint8, device=cuda)
    sums = torch.zeros(16, device=cuda)
    with pytest.raises(pg.PgError):
        pg.selftest_training_waits(scratch[4:], sums)  # misaligned
    with pytest.raises(pg.PgError):
        pg.selftest_training_waits(scratch, sums[1:])
    with pytest.raises(ValueError):
        pg.selftest_training_waits(scratch[:2000], sums)
    with pytest.raises(ValueError):
        pg.selftest_training_waits(scratch, sums[:7])
