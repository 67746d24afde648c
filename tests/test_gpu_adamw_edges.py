"""Edges of dm_adamw_step on the GPU: remainders next to the rounding's noise,
the least and the largest eps."""
import numpy as np
import pytest
import torch

import dimuon_optimizer_b200 as dm
from gpu_harness import to_host
from oracle import adamw_oracle as ao
from test_gpu_adamw import check_fp32, workspace

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

F32 = np.float32


def codes(t):
    return t.view(torch.uint8).cpu().numpy()


def test_subnormal_codes_round_by_their_whole_remainder():
    """With both betas 0 and zero states the new moments are g and g^2.  Each
    subnormal value lies just below j + k / 65536 steps of its code, where the
    element's noise is 1 - k / 65536: remainder and noise stay below one, so
    the code is j.  (The remainder rounded to 20 or 21 bits first gives j + 1.)"""
    n, seed, t = 1 << 14, 5, 9
    rng = np.random.default_rng(41)
    u1, u2 = ao.noise(seed, t, 0, n)
    # first moment: steps of 2^-9 beside a largest value of 448
    k = 1.0 - u1
    G1 = ((rng.integers(0, 4, n) + k - 2.0 ** -22) * 2.0 ** -9).astype(F32)
    # second moment: steps of 2^-16 beside one just below 57344, the square of a gradient next to the root
    target = (1 + (1.0 - u2) - 2.0 ** -23) * 2.0 ** -16
    root = np.sqrt(target).astype(F32)
    tries = [root]
    for d in (-np.inf, np.inf):
        x = root
        for _ in range(3):
            x = np.nextafter(x, F32(d))
            tries.append(x)
    G2 = root.copy()
    for x in tries:
        G2 = np.where((x * x).astype(np.float64) == target, x, G2)
    hit = (G2 * G2).astype(np.float64) == target
    hit[::128] = False
    assert hit.sum() > 1000
    G1[::128], G2[::128] = 448.0, np.nextafter(F32(np.sqrt(57344.0)), F32(0))
    hp = dm.dm_adamw_default_hparams(beta1=0.0, beta2=0.0, seed=seed, step=t)
    for which, G in ((0, G1), (1, G2)):
        W = torch.zeros(n, device="cuda")
        st = dm.dm_adamw_state(W, dm.DM_STATE_8BIT)
        ts = [dm.dm_adamw_tensor(W, torch.from_numpy(G).cuda(), *st)]
        dm.check(dm.dm_adamw_step(ts, hp, workspace(ts, hp)))
        c1, s1, c2, s2 = ao.pack_moments(G.astype(float), (G * G).astype(float), seed, t, 0)
        if which == 0:
            body = np.arange(n) % 128 != 0
            want = np.floor(G[body].astype(float) * 2.0 ** 9)  # j, by construction
            assert (s1 == 1).all() and np.array_equal(c1[body], want)
        else:
            assert (s2 == 1).all() and (c2[hit] == 1).all()
        np.testing.assert_array_equal(to_host(st[2]), s1)
        np.testing.assert_array_equal(to_host(st[3]), s2)
        np.testing.assert_array_equal(codes(st[0]), c1)
        np.testing.assert_array_equal(codes(st[1]), c2)


@pytest.mark.parametrize("state", [dm.DM_STATE_FP32, dm.DM_STATE_8BIT])
@pytest.mark.parametrize("eps", [2.0 ** -126, 2.0 ** 125])
def test_zero_gradients_at_the_limits_of_eps(state, eps):
    """Elements that saw no gradient divide 0 by eps alone; the others follow the formula."""
    n = 3000
    rng = np.random.default_rng(42)
    W0, G = rng.standard_normal((2, n)).astype(F32)
    G[::3] = 0
    W = torch.from_numpy(W0).cuda()
    hp = dm.dm_adamw_default_hparams(eps=eps, weight_decay=0.0)
    ts = [dm.dm_adamw_tensor(W, torch.from_numpy(G).cuda(), *dm.dm_adamw_state(W, state))]
    dm.check(dm.dm_adamw_step(ts, hp, workspace(ts, hp)))
    z = np.zeros(n)
    check_fp32(W0.astype(float), G.astype(float), z, z, hp, 1, to_host(W), None, None, torch.float32)
    assert np.array_equal(to_host(W)[::3], W0[::3])
