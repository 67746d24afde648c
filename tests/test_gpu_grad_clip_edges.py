"""dm_grad_clip on the GPU: what its bits depend on, and README's training step."""
import os
import re

import numpy as np
import pytest
import torch

import dimuon_optimizer_b200 as dm
from conftest import ROOT
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


def test_readme_step_leaves_everything_where_a_gradient_is_nan():
    """README's example as it stands: a step that moves all weights, then one
    with a NaN in one of Muon's gradients, which moves none and no state."""
    with open(os.path.join(ROOT, "README.md")) as fh:
        muon, both = re.findall(r"```python\n(.*?)```", fh.read(), re.S)
    torch.manual_seed(52)
    muon_w = [torch.randn(s, device="cuda").to(BF) for s in ((64, 96), (96, 64))]
    muon_grads = [torch.randn_like(w) for w in muon_w]
    momenta = [torch.zeros(w.shape, device="cuda") for w in muon_w]
    other_weights = [torch.randn(s, device="cuda").to(BF) for s in ((50, 64), (333,))]
    other_grads = [torch.randn_like(w) for w in other_weights]
    rows, cols = muon_w[0].shape
    env = {"W": muon_w[0], "G": muon_grads[0], "M": momenta[0],
           "row_energy": torch.zeros(rows, device="cuda"), "col_energy": torch.zeros(cols, device="cuda"),
           "muon_grads": muon_grads, "other_weights": other_weights, "other_grads": other_grads}
    exec(muon, env)  # one Dimuon step over the first matrix
    env["mats"] = [dm.dm_matrix(*x) for x in zip(muon_w, muon_grads, momenta)]
    env["ws"] = torch.empty(dm.dm_workspace_size(env["mats"], env["hp"], 0), dtype=torch.uint8,
                            device="cuda")
    setup, step = both.split("dm.check(dm.dm_grad_clip", 1)
    exec("import torch, dimuon_optimizer_b200 as dm\n" + setup, env)
    step = "dm.check(dm.dm_grad_clip" + step

    def state():
        return [t.clone() for t in muon_w + momenta + other_weights
                + [x.view(torch.uint8) for d in env["ts"]._keep for x in d[2:]]]

    before = state()
    exec(step, env)
    after = state()
    assert not any(torch.equal(a, b) for a, b in zip(before, after)) and env["count"].item() == 1
    muon_grads[1][3, 5] = float("nan")
    exec(step, env)
    assert all(torch.equal(a, b) for a, b in zip(after, state())) and env["count"].item() == 1
