"""Pins of the many-tensor operators' oracle (oracle/adamw_oracle.py) against
other sources: torch's AdamW in float64, torch's float8 formats, exact
expectations of the stochastic rounding."""
import numpy as np
import pytest
import torch

from oracle import adamw_oracle as ao


@pytest.mark.parametrize("wd", [0.0, 0.1])
def test_step_is_torchs_adamw(wd):
    rng = np.random.default_rng(1)
    w0 = rng.standard_normal(50)
    p = torch.nn.Parameter(torch.from_numpy(w0.copy()))
    hp = ao.AdamWParams(lr=0.0078125, beta1=0.875, beta2=0.9921875, eps=2.0 ** -20,
                        weight_decay=np.float32(wd))  # exact in float32
    opt = torch.optim.AdamW([p], lr=hp.lr, betas=(hp.beta1, hp.beta2), eps=hp.eps,
                            weight_decay=float(hp.weight_decay))
    w, m, v = w0, np.zeros(50), np.zeros(50)
    for t in range(1, 6):
        g = rng.standard_normal(50)
        p.grad = torch.from_numpy(g.copy())
        opt.step()
        r = ao.adamw_step(w, g, m, v, hp, t)
        w, m, v = r.W, r.m, r.v
        # both in float64; a step rounds some 10 times, each at most 2^-53
        np.testing.assert_allclose(w, p.detach().numpy(), rtol=5 * 20 * 2.0 ** -53,
                                   atol=5 * 20 * 2.0 ** -53)


def test_multipliers_and_scale():
    rng = np.random.default_rng(2)
    w, g, m = rng.standard_normal((3, 20))
    v = rng.random(20)
    hp = ao.AdamWParams(lr=0.5, weight_decay=0.25)
    a = ao.adamw_step(w, g, m, v, hp, 3, grad_scale=0.5, lr_mult=0.25, decay_mult=2.0)
    b = ao.adamw_step(w, 0.5 * g, m, v, ao.AdamWParams(lr=0.125, weight_decay=0.5), 3)
    for x, y in ((a.W, b.W), (a.m, b.m), (a.v, b.v)):
        np.testing.assert_array_equal(x, y)


@pytest.mark.parametrize("table,dtype", [(ao.E4M3, torch.float8_e4m3fn),
                                         (ao.E5M2, torch.float8_e5m2)])
def test_formats_are_torchs(table, dtype):
    codes = torch.arange(len(table), dtype=torch.uint8)
    np.testing.assert_array_equal(codes.view(dtype).double().numpy(), table)
    assert table[-1] == torch.finfo(dtype).max


def test_block_scales():
    for top in (448.0, 57344.0):
        for a, want in ((top, 1.0), (np.nextafter(top, 1e9), 2.0), (top / 2, 0.5),
                        (np.nextafter(top / 2, 1e9), 1.0), (0.0, 2.0 ** -110),
                        (1e-45, 2.0 ** -110)):
            x = np.zeros(200)
            x[130] = -a
            np.testing.assert_array_equal(ao.block_scales(x, top), [2.0 ** -110, want])


@pytest.mark.parametrize("table", [ao.E4M3, ao.E5M2])
def test_stochastic_rounding_is_unbiased(table):
    """Over all 65536 noise values the mean of the codes' values is x up to the
    noise's own step (u is a multiple of 2^-16, so the probability of the upper
    neighbour is the remainder up to 2^-16)."""
    u = np.arange(65536) / 65536
    for i, frac in ((0, 0.3), (1, 0.001), (7, 0.5), (40, 0.9991), (len(table) - 2, 0.25)):
        gap = table[i + 1] - table[i]
        x = table[i] + frac * gap
        c = ao.stochastic_codes(np.full(65536, x), np.ones(512), table, u)
        assert set(c) <= {i, i + 1}
        assert abs(table[c].mean() - x) <= gap * 2.0 ** -16
    # values on the grid stay, whatever the noise
    for i in (0, 3, len(table) - 1):
        c = ao.stochastic_codes(np.full(65536, table[i]), np.ones(512), table, u)
        assert (c == i).all()


def test_pack_keeps_small_second_moments_positive():
    v = np.full(128, 1e-30)
    v[0] = 1.0
    _, _, c2, s2 = ao.pack_moments(v, v, 5, 1, 0)
    assert (c2 > 0).all() and s2[0] > 0


def test_noise_is_uniform_and_differs():
    """Means and correlations of the noise within five standard errors
    (uniform on [0, 1): variance 1/12), between the moments, neighbouring
    elements, steps, tensors and seeds."""
    n = 1 << 16
    a1, a2 = ao.noise(7, 100, 3, n)
    se = np.sqrt(1 / 12 / n)
    for u in (a1, a2):
        assert abs(u.mean() - 0.5) < 5 * se and u.min() >= 0 and u.max() < 1
    others = [a2, np.roll(a1, 1), np.roll(a1, 16), ao.noise(7, 101, 3, n)[0],
              ao.noise(7, 100, 4, n)[0], ao.noise(8, 100, 3, n)[0]]
    for u in others:
        c = ((a1 - 0.5) * (u - 0.5)).mean() * 12
        assert abs(c) < 5 / np.sqrt(n)
    # any range of a tensor has the noise of its elements
    b1, _ = ao.noise(7, 100, 3, 100, first=1000)
    np.testing.assert_array_equal(b1, a1[1000:1100])


def test_second_moment_follows_where_nearest_rounding_stands_still():
    """The reason for the stochastic rounding: gradients whose size falls to a
    third.  v must fall to a ninth; nearest rounding keeps it where it was."""
    rng = np.random.default_rng(3)
    hp = ao.AdamWParams()
    n = 128 * 16
    v = np.full(n, 1.0)
    near = np.full(n, 1.0)
    # the anchor keeps each block's scale (and its weight in the mean is removed)
    for t in range(1, 4001):
        g = rng.standard_normal(n) / 3
        g[::128] = 4.0
        v = f = hp.beta2 * v + (1 - hp.beta2) * g * g
        c, s = None, ao.block_scales(f, 57344.0)
        _, u2 = ao.noise(1, t, 0, n)
        c = ao.stochastic_codes(f, s, ao.E5M2, u2)
        v = ao.unpack(c, s, ao.E5M2)
        q = hp.beta2 * near + (1 - hp.beta2) * g * g
        s = ao.block_scales(q, 57344.0)
        near = ao.unpack(ao.stochastic_codes(q, s, ao.E5M2, np.full(n, 0.5)), s, ao.E5M2)
    body = np.ones(n, bool)
    body[::128] = False
    # after 4000 steps the start has decayed to exp(-4): expected 1/9 + 8/9 e^-4 = 0.127;
    # one element's spread is about a third of it, so the mean of 2032 is within 5 %
    assert abs(v[body].mean() / 0.1274 - 1) < 0.05
    assert near[body].mean() > 0.5


def test_grad_clip_against_torch():
    rng = np.random.default_rng(4)
    grads = [rng.standard_normal(k) for k in (1, 0, 7, 300)]
    ps = [torch.nn.Parameter(torch.zeros(len(g), dtype=torch.float64)) for g in grads]
    for p, g in zip(ps, grads):
        p.grad = torch.from_numpy(g.copy())
    for limit in (0.5, 1e9):
        want = torch.nn.utils.get_total_norm([p.grad for p in ps])
        norm, c, _ = ao.grad_clip(grads, limit)
        assert norm == pytest.approx(float(want), rel=1e-14)
        assert c == pytest.approx(min(1.0, limit / norm), rel=1e-15)
    assert ao.grad_clip([np.zeros(4)], 1.0)[:2] == (0.0, 1.0)
