"""Edges of dm_adamw_step on the GPU: remainders next to the rounding's noise,
the least and the largest eps, moments at the end of fp32's range,
steps over no elements."""
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


def big_gradients(n, seed):
    """Ordinary gradients, and in every fourth block of 128 one whose square overflows."""
    rng = np.random.default_rng(seed)
    G = rng.standard_normal(n).astype(F32)
    at = np.arange(37, n, 512)
    G[at] = rng.choice([1e20, -3e25, 2e19, 3e38], len(at))
    return G, at


@pytest.mark.parametrize("shift", [0, 1])
def test_a_finite_gradient_leaves_finite_8bit_moments(shift):
    """Gradients above 1.8e19 square to infinity in fp32.  Their blocks stay
    finite over the steps that follow: codes, scales and weights as the oracle's
    (the element itself moves by m / infinity, nothing, in the first step)."""
    n, seed = 3000, 13
    rng = np.random.default_rng(43)
    W = torch.zeros(n + shift, device="cuda")[shift:]
    W.copy_(torch.from_numpy(rng.standard_normal(n)))
    st = dm.dm_adamw_state(W, dm.DM_STATE_8BIT)
    hp = dm.dm_adamw_default_hparams(seed=seed, weight_decay=0.0)
    p = ao.AdamWParams(hp.lr, hp.beta1, hp.beta2, hp.eps, hp.weight_decay)
    g = torch.zeros(n, device="cuda")
    ts = [dm.dm_adamw_tensor(W, g, *st)]
    ws = workspace(ts, hp)
    m0 = v0 = np.zeros(n)
    for t in (1, 2, 3):
        G, at = big_gradients(n, 44) if t == 1 else (rng.standard_normal(n).astype(F32), None)
        g.copy_(torch.from_numpy(G))
        hp.step = t
        w0 = to_host(W)
        dm.check(dm.dm_adamw_step(ts, hp, ws))
        assert torch.isfinite(W).all() and all(torch.isfinite(s).all() for s in st[2:])
        if t == 1:  # what overflows moves by nothing, the rest by the formula
            assert np.array_equal(to_host(W)[at], w0[at])
        keep = np.ones(n, bool)
        keep[at if t == 1 else []] = False
        check_fp32(w0[keep], G[keep].astype(float), m0[keep], v0[keep], hp, t, to_host(W)[keep], None,
                   None, torch.float32)
        m32, v32 = ao.moments_f32(G, m0, v0, p)
        assert np.isinf(v32).any() == (t == 1) and np.isfinite(m32).all()
        c1, s1, c2, s2 = ao.pack_moments(m32.astype(float), v32.astype(float), seed, t, 0)
        np.testing.assert_array_equal(to_host(st[2]), s1)
        np.testing.assert_array_equal(to_host(st[3]), s2)
        np.testing.assert_array_equal(codes(st[0]), c1)
        np.testing.assert_array_equal(codes(st[1]), c2)
        m0, v0 = ao.unpack(c1, s1, ao.E4M3), ao.unpack(c2, s2, ao.E5M2)


def test_a_finite_gradient_in_fp32_moments():
    """The same with fp32 moments: infinite in that element alone, which stays
    where it is; its neighbours go on."""
    n = 3000
    W0 = torch.randn(n, device="cuda")
    W = W0.clone()
    G, at = big_gradients(n, 44)
    g = torch.from_numpy(G).cuda()
    m, v = dm.dm_adamw_state(W)
    hp = dm.dm_adamw_default_hparams(weight_decay=0.0)
    ts = [dm.dm_adamw_tensor(W, g, m, v)]
    for t in (1, 2, 3):
        hp.step = t
        dm.check(dm.dm_adamw_step(ts, hp, workspace(ts, hp)))
        g.normal_()
    hit = torch.zeros(n, dtype=torch.bool, device="cuda")
    hit[torch.from_numpy(at).cuda()] = True
    assert torch.equal(W[hit], W0[hit]) and torch.isinf(v[hit]).all() and torch.isfinite(m).all()
    assert torch.isfinite(W).all() and torch.isfinite(v[~hit]).all() and (W[~hit] != W0[~hit]).all()


def test_moments_at_the_end_of_fp32():
    """Moments between 1.75 x 2^127 and fp32's end (both betas 0: g and g^2):
    second ones are stored as 1.75 x 2^127, not rounded up to 2^128."""
    n = 4096
    for G in (np.linspace(2.9e38, 3.4e38, n), np.linspace(1.7e19, 1.8446743e19, n)):
        G = G.astype(F32)
        G[::2] *= -1
        W = torch.zeros(n, device="cuda")
        st = dm.dm_adamw_state(W, dm.DM_STATE_8BIT)
        hp = dm.dm_adamw_default_hparams(beta1=0.0, beta2=0.0, seed=3)
        ts = [dm.dm_adamw_tensor(W, torch.from_numpy(G).cuda(), *st)]
        dm.check(dm.dm_adamw_step(ts, hp, workspace(ts, hp)))
        with np.errstate(over="ignore"):
            c1, s1, c2, s2 = ao.pack_moments(G.astype(float), (G * G).astype(float), 3, 1, 0)
        for got, want in zip(st, (c1, c2, s1, s2)):
            np.testing.assert_array_equal(codes(got) if got.element_size() == 1 else to_host(got), want)
        assert (st[1].float() * st[3].repeat_interleave(128)).max().item() == ao.LARGEST


@pytest.mark.parametrize("which", ["grad_scale", "lr_dev"])
@pytest.mark.parametrize("counted", [False, True])
def test_a_step_over_no_elements_reports_its_device_values(which, counted):
    value = torch.tensor([float("nan")], device="cuda")
    count = torch.tensor([4], dtype=torch.int64, device="cuda")
    hp = dm.dm_adamw_default_hparams(**{which: value}, **({"step_counter": count} if counted else {}))
    empty = [dm.dm_adamw_tensor(*(torch.zeros(0, device="cuda") for _ in range(4)))]
    for ts in ([], empty):
        value.fill_(float("nan"))
        ws = workspace(ts, hp)
        dm.check(dm.dm_adamw_step(ts, hp, ws))
        assert dm.dm_read_device_status(ws) == dm.DM_ERR_NONFINITE and count.item() == 4
        value.fill_(0.5)
        dm.check(dm.dm_adamw_step(ts, hp, ws))
        assert dm.dm_read_device_status(ws) == dm.DM_OK and count.item() == (5 if counted else 4)
        count.fill_(4)
