"""dm_grad_clip on the GPU: what its bits depend on."""
import numpy as np
import pytest
import torch

import dimuon_optimizer_b200 as dm
from test_gpu_adamw import BF, F32, U, Buf
from test_gpu_grad_clip import call

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


@pytest.mark.parametrize("gdt", [BF, F32])
def test_buffers_that_lie_alike_give_the_same_bits(gdt):
    """The same values at offsets equal modulo 16 elements; at any other the
    norm is within its tolerance twice."""
    rng = np.random.default_rng(51)
    lists = [[rng.standard_normal(n) for n in lengths]
             for lengths in ((1,), (16,), (33,), (20, 47), (100, 7, 1025), (16384 + 9, 3, 70001))] + \
        [[rng.standard_normal(int(n))] for n in rng.integers(17, 200, 40)]
    for vals in lists:
        shifts = rng.integers(0, 16, len(vals))

        def norm(more):
            bufs = [Buf(len(v), gdt, int(s) + more, v) for v, s in zip(vals, shifts)]
            return call([dm.dm_grad_tensor(b.t) for b in bufs], 0.5)

        first = norm(0)
        for more in (16, 48, 64):
            assert torch.equal(norm(more), first)
        other = norm(5)
        assert abs(other[0].item() - first[0].item()) <= 20 * U * first[0].item()
