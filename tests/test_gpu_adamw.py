"""dm_adamw_step on the GPU against the fp64 oracle (oracle/adamw_oracle.py).

Tolerances (u = 2^-24, half a unit of fp32 relative to the value):
  m': the gradient's scaling, (1 - b1) rounded to fp32, two products and a sum
      round once each: |err| <= 5 u (|b1 m| + |(1 - b1) g|).
  v': as m', with the gradient's rounding twice and one for its square:
      |err| <= 7 u v' (all terms are positive).
  update = step m' / d: what m' is off, divided by d, and relative errors of d
      (v': 3.5 u; square root 2 u (sqrt.approx, 2^-23); the bias correction
      and its product 2 u; sum 1 u), of the division (2 ulp: 4 u) and of step
      (lr times multiplier, bias correction, product: 3 u): below 16 u.
  W': decay coefficient and two roundings of the sum, 3 u (|W| + |update|), then
      half a storage step, eps / 2 |W'| (bf16 2^-8, fp32 2^-24).
  Absolute floors of 2^-140 stand for what underflows.
8-bit codes and scales are compared exactly with the oracle's, from the
moments as fp32 products and sums rounded one by one (their definition).
"""
import numpy as np
import pytest
import torch

import dimuon_optimizer_b200 as dm
from gpu_harness import to_host
from oracle import adamw_oracle as ao

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
SENTINEL = 37.0  # exact in every type used, 8-bit floats through their bytes
PAD = 64


class Buf:
    """`n` elements at element offset `shift` of a 256-byte aligned buffer,
    with a guard of PAD + shift elements around them."""

    def __init__(self, n, dtype, shift=0, fill=None):
        self.raw = torch.full((n + 2 * PAD + shift,), 37, dtype=torch.uint8, device="cuda").view(dtype) \
            if dtype.itemsize == 1 else torch.full((n + 2 * PAD + shift,), SENTINEL, dtype=dtype,
                                                   device="cuda")
        self.t = self.raw[PAD + shift:PAD + shift + n]
        self.lo, self.hi = PAD + shift, PAD + shift + n
        if fill is not None:
            self.t.copy_(torch.as_tensor(fill))

    def check(self):
        ints = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[self.raw.element_size()]
        want = torch.full((1,), SENTINEL, dtype=self.raw.dtype).view(ints) \
            if self.raw.element_size() > 1 else torch.tensor([37], dtype=torch.uint8)
        r = self.raw.view(ints)
        for part in (r[:self.lo], r[self.hi:]):
            assert (part == want.to("cuda")).all(), "written outside the tensor"


def workspace(tensors, hp):
    return torch.full((dm.dm_adamw_workspace_size(tensors, hp),), 0xFF, dtype=torch.uint8,
                      device="cuda")


def draw(n, seed):
    """(W, G, m, v) with gradients over several decades, zeros among them."""
    rng = np.random.default_rng(seed)
    size = np.exp(3 * rng.standard_normal(n))
    G = rng.standard_normal(n) * size * (rng.random(n) > 0.1)
    return (0.5 * rng.standard_normal(n), G, 0.3 * rng.standard_normal(n) * size,
            size ** 2 * (0.1 + rng.random(n)))


def check_fp32(W0, G, m0, v0, hp, t, W, M, V, wdt, gs=1.0, lr_mult=1.0, decay_mult=1.0):
    """Compares new (W, M, V) with the oracle's, from the stored inputs."""
    p = ao.AdamWParams(hp.lr, hp.beta1, hp.beta2, hp.eps, hp.weight_decay)
    r = ao.adamw_step(W0, G, m0, v0, p, t, grad_scale=gs, lr_mult=lr_mult, decay_mult=decay_mult)
    b1, b2 = float(np.float32(hp.beta1)), float(np.float32(hp.beta2))
    g = G * float(np.float32(gs))
    tiny = 2.0 ** -140
    em = 5 * U * (np.abs(b1 * m0) + np.abs((1 - b1) * g)) + tiny
    if M is not None:
        assert np.all(np.abs(M - r.m) <= em)
        assert np.all(np.abs(V - r.v) <= 7 * U * r.v + tiny)
    lr = float(np.float32(hp.lr)) * lr_mult
    d = np.sqrt(r.v / (1 - b2 ** t)) + hp.eps
    eu = 16 * U * np.abs(r.update) + lr / (1 - b1 ** t) * em / np.maximum(d, 1e-30)
    half = torch.finfo(wdt).eps / 2
    tol = eu + 3 * U * (np.abs(W0) + np.abs(r.update))
    tol = tol + half * (np.abs(r.W) + tol) + tiny
    bad = np.abs(W - r.W) > tol
    assert not bad.any(), (np.abs(W - r.W)[bad][:4], tol[bad][:4], np.nonzero(bad)[0][:4])


SIZES = [1, 2, 7, 8, 9, 15, 16, 17, 127, 128, 129, 500, 2047, 2048, 2049, 4095, 4096, 4097, 10007]


@pytest.mark.parametrize("wdt", [BF, F32])
@pytest.mark.parametrize("gdt", [BF, F32])
@pytest.mark.parametrize("layout", ["aligned", "same_offset", "mixed_offset"])
def test_fp32_moments(wdt, gdt, layout):
    hp = dm.dm_adamw_default_hparams(lr=3e-3, weight_decay=0.1, step=3)
    bufs, host, ts = [], [], []
    for i, n in enumerate(SIZES + [0]):
        W, G, m, v = draw(n, i)
        s = [0] * 4 if layout == "aligned" else [i % 8] * 4 if layout == "same_offset" else \
            [(i + k * 3) % 8 for k in range(4)]
        b = [Buf(n, dt, sh, x) for x, dt, sh in zip((W, G, m, v), (wdt, gdt, F32, F32), s)]
        bufs.append(b)
        host.append([to_host(x.t) for x in b])
        ts.append(dm.dm_adamw_tensor(*(x.t for x in b), lr_mult=1.0 - 0.1 * (i % 3),
                                     decay_mult=float(i % 2)))
    gs = torch.tensor([0.25], device="cuda")
    hp = dm.dm_adamw_default_hparams(lr=3e-3, weight_decay=0.1, step=3, grad_scale=gs)
    ws = workspace(ts, hp)
    dm.check(dm.dm_adamw_step(ts, hp, ws))
    assert dm.dm_read_device_status(ws) == dm.DM_OK
    for i, (b, h) in enumerate(zip(bufs, host)):
        for x in b:
            x.check()
        assert np.array_equal(to_host(b[1].t), h[1])  # the gradient stays
        check_fp32(*h, hp, 3, to_host(b[0].t), to_host(b[2].t), to_host(b[3].t), wdt, 0.25,
                   float(np.float32(1.0 - 0.1 * (i % 3))), float(i % 2))


@pytest.mark.parametrize("wdt,gdt", [(BF, BF), (F32, F32), (F32, BF), (BF, F32)])
@pytest.mark.parametrize("shift", [0, 3])
def test_8bit_moments(wdt, gdt, shift):
    """Codes and scales equal the oracle's, over three steps from zero."""
    gs = torch.tensor([0.5], device="cuda")
    hp = dm.dm_adamw_default_hparams(lr=3e-3, weight_decay=0.1, seed=1234, grad_scale=gs)
    p = ao.AdamWParams(hp.lr, hp.beta1, hp.beta2, hp.eps, hp.weight_decay)
    bufs, ts = [], []
    for i, n in enumerate(SIZES + [0]):
        blocks = -(-n // 128)
        W, G, _, _ = draw(n, 100 + i)
        b = [Buf(n, wdt, shift, W), Buf(n, gdt, shift, G), Buf(n, torch.float8_e4m3fn, shift),
             Buf(n, torch.float8_e5m2, shift), Buf(blocks, F32, 0, np.zeros(blocks)),
             Buf(blocks, F32, 0, np.zeros(blocks))]
        for x in b[2:4]:
            x.t.view(torch.uint8).zero_()
        bufs.append(b)
        ts.append(dm.dm_adamw_tensor(*(x.t for x in b)))
    ws = workspace(ts, hp)
    for t in (1, 2, 3):
        hp.step = t
        for i, b in enumerate(bufs):
            b[1].t.copy_(torch.from_numpy(draw(b[1].t.numel(), 1000 * t + i)[1]))
        before = []
        for b in bufs:
            c1, c2 = (x.t.view(torch.uint8).cpu().numpy() for x in b[2:4])
            s1, s2 = (to_host(x.t) for x in b[4:6])
            before.append((to_host(b[0].t), to_host(b[1].t), ao.unpack(c1, s1, ao.E4M3),
                           ao.unpack(c2, s2, ao.E5M2)))
        dm.check(dm.dm_adamw_step(ts, hp, ws))
        assert dm.dm_read_device_status(ws) == dm.DM_OK
        for i, (b, h) in enumerate(zip(bufs, before)):
            for x in b:
                x.check()
            m32, v32 = ao.moments_f32(h[1], h[2], h[3], p, 0.5)
            c1, s1, c2, s2 = ao.pack_moments(m32.astype(np.float64), v32.astype(np.float64),
                                             1234, t, i)
            np.testing.assert_array_equal(to_host(b[4].t), s1)
            np.testing.assert_array_equal(to_host(b[5].t), s2)
            np.testing.assert_array_equal(b[2].t.view(torch.uint8).cpu().numpy(), c1)
            np.testing.assert_array_equal(b[3].t.view(torch.uint8).cpu().numpy(), c2)
            check_fp32(*h, hp, t, to_host(b[0].t), None, None, wdt, 0.5)


def test_8bit_blocks_of_extreme_range():
    """Blocks whose largest gradient is 1e18 .. 1e-19, with far smaller ones
    beside it: codes and scales as the oracle's, positive second moments above zero."""
    rng = np.random.default_rng(21)
    tops = [1e18, 1e15, 1e12, 1e9, 1e6, 1.0, 1e-9, 1e-15, 1e-19]
    G = []
    for top in tops:
        b = rng.standard_normal(128) * top * 10.0 ** -rng.uniform(0, 22, 128)
        b[rng.integers(128)] = top
        b[rng.integers(1, 128)] = 0.0
        G.append(b)
    G = np.concatenate(G).astype(np.float32)
    W = torch.zeros(len(G), device="cuda")
    g = torch.from_numpy(G).cuda()
    st = dm.dm_adamw_state(W, dm.DM_STATE_8BIT)
    hp = dm.dm_adamw_default_hparams(seed=2)
    p = ao.AdamWParams(hp.lr, hp.beta1, hp.beta2, hp.eps, hp.weight_decay)
    ts = [dm.dm_adamw_tensor(W, g, *st)]
    ws = workspace(ts, hp)
    z = np.zeros(len(G))
    h = (z, z)
    for t in (1, 2):
        hp.step = t
        dm.check(dm.dm_adamw_step(ts, hp, ws))
        m32, v32 = ao.moments_f32(G, *h, p)
        c1, s1, c2, s2 = ao.pack_moments(m32.astype(float), v32.astype(float), 2, t, 0)
        np.testing.assert_array_equal(to_host(st[2]), s1)
        np.testing.assert_array_equal(to_host(st[3]), s2)
        np.testing.assert_array_equal(st[0].view(torch.uint8).cpu().numpy(), c1)
        np.testing.assert_array_equal(st[1].view(torch.uint8).cpu().numpy(), c2)
        assert ((c2 > 0) == (v32 > 0)).all()
        h = (ao.unpack(c1, s1, ao.E4M3), ao.unpack(c2, s2, ao.E5M2))


@pytest.mark.parametrize("wdt,gdt", [(BF, BF), (F32, F32)])
def test_moments_are_rounded_product_by_product(wdt, gdt):
    """The new moments' bits are those of separate fp32 products and sums (a
    multiply-add in their place changes a quarter of them), and so are the
    8-bit codes, also where a block's largest moment lies at a scale's border."""
    n = 1 << 18
    rng = np.random.default_rng(31)
    gs = torch.tensor([0.37], device="cuda")
    hp = dm.dm_adamw_default_hparams(grad_scale=gs, step=5, seed=8)
    p = ao.AdamWParams(hp.lr, hp.beta1, hp.beta2, hp.eps, hp.weight_decay)
    W, G = (torch.from_numpy(rng.standard_normal(n)).float().cuda() for _ in "wg")
    W, G = W.to(wdt), G.to(gdt)
    m, v = (torch.from_numpy(x).float().cuda() for x in (rng.standard_normal(n), rng.random(n)))
    h = [to_host(x) for x in (G, m, v)]
    ts = [dm.dm_adamw_tensor(W, G, m, v)]
    dm.check(dm.dm_adamw_step(ts, hp, workspace(ts, hp)))
    m32, v32 = ao.moments_f32(*h, p, 0.37)
    assert np.array_equal(to_host(m), m32) and np.array_equal(to_host(v), v32)
    st = dm.dm_adamw_state(W, dm.DM_STATE_8BIT)
    st[0].view(torch.uint8).copy_(torch.from_numpy(rng.integers(0, 127, n, dtype=np.uint8)))
    st[1].view(torch.uint8).copy_(torch.from_numpy(rng.integers(0, 124, n, dtype=np.uint8)))
    st[2].fill_(2.0 ** -9)
    st[3].fill_(2.0 ** -17)
    before = (ao.unpack(st[0].view(torch.uint8).cpu().numpy(), to_host(st[2]), ao.E4M3),
              ao.unpack(st[1].view(torch.uint8).cpu().numpy(), to_host(st[3]), ao.E5M2))
    ts = [dm.dm_adamw_tensor(W, G, *st)]
    dm.check(dm.dm_adamw_step(ts, hp, workspace(ts, hp)))
    m32, v32 = ao.moments_f32(h[0], *before, p, 0.37)
    c1, s1, c2, s2 = ao.pack_moments(m32.astype(float), v32.astype(float), 8, 5, 0)
    np.testing.assert_array_equal(to_host(st[2]), s1)
    np.testing.assert_array_equal(to_host(st[3]), s2)
    np.testing.assert_array_equal(st[0].view(torch.uint8).cpu().numpy(), c1)
    np.testing.assert_array_equal(st[1].view(torch.uint8).cpu().numpy(), c2)


def test_many_tensors_and_both_states_in_one_call():
    """More tensors than one launch holds, the two state formats mixed; the
    8-bit noise goes by the position in the call."""
    rng = np.random.default_rng(5)
    hp = dm.dm_adamw_default_hparams(seed=9, step=2)
    p = ao.AdamWParams(hp.lr, hp.beta1, hp.beta2, hp.eps, hp.weight_decay)
    items, ts = [], []
    for i in range(1000):
        n = int(rng.integers(0, 300))
        W, G, m, v = (torch.from_numpy(x).float().cuda() for x in draw(n, 2000 + i))
        st = (m, v) if i % 3 else dm.dm_adamw_state(W, dm.DM_STATE_8BIT)
        items.append((n, W, G, st))
        ts.append(dm.dm_adamw_tensor(W, G, *st))
    host = [(to_host(W), to_host(G), to_host(st[0]), to_host(st[1])) for _, W, G, st in items]
    arr = dm.dm_adamw_tensors(ts)
    ws = workspace(arr, hp)
    dm.check(dm.dm_adamw_step(arr, hp, ws))
    for i, ((n, W, G, st), h) in enumerate(zip(items, host)):
        eight = len(st) == 4
        check_fp32(*h, hp, 2, to_host(W), None if eight else to_host(st[0]),
                   None if eight else to_host(st[1]), F32)
        if eight and n:
            m32, v32 = ao.moments_f32(h[1], h[2], h[3], p)
            c1, s1, c2, s2 = ao.pack_moments(m32.astype(float), v32.astype(float), 9, 2, i)
            np.testing.assert_array_equal(st[0].view(torch.uint8).cpu().numpy(), c1)
            np.testing.assert_array_equal(st[1].view(torch.uint8).cpu().numpy(), c2)


@pytest.mark.parametrize("state", [dm.DM_STATE_FP32, dm.DM_STATE_8BIT])
@pytest.mark.parametrize("which", ["grad_scale", "lr_dev"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("counted", [False, True])
def test_a_non_finite_device_value_skips_the_step(state, which, bad, counted):
    W = torch.randn(5000, device="cuda").to(BF)
    G = torch.randn(5000, device="cuda")
    st = dm.dm_adamw_state(W, state)
    value = torch.tensor([bad], device="cuda")
    counter = torch.tensor([4], dtype=torch.int64, device="cuda")
    more = {"step_counter": counter} if counted else {}
    hp = dm.dm_adamw_default_hparams(**{which: value}, **more)
    ts = [dm.dm_adamw_tensor(W, G, *st)]
    ws = workspace(ts, hp)
    before = [x.clone() for x in (W, *(s.view(torch.uint8) for s in st))]
    dm.check(dm.dm_adamw_step(ts, hp, ws))
    assert dm.dm_read_device_status(ws) == dm.DM_ERR_NONFINITE
    for a, b in zip(before, (W, *(s.view(torch.uint8) for s in st))):
        assert torch.equal(a, b)
    assert counter.item() == 4
    # the next step with a finite value runs and clears the status
    value.fill_(0.5)
    dm.check(dm.dm_adamw_step(ts, hp, ws))
    assert dm.dm_read_device_status(ws) == dm.DM_OK
    assert not torch.equal(before[0], W)
    assert counter.item() == (5 if counted else 4)


def test_non_finite_gradients_stay_where_they_are():
    """Without clipping: fp32 moments carry NaN in that element only; 8-bit
    ones in its block of 128 (a NaN scale), the other blocks as without it."""
    n = 1000
    rng = np.random.default_rng(6)
    W0, G0 = (torch.from_numpy(rng.standard_normal(n)).float().cuda() for _ in "wg")
    for bad in (float("nan"), float("inf")):
        G1 = G0.clone()
        G1[300] = bad
        res = []
        for G in (G0, G1):
            W = [W0.clone(), W0.clone()]
            st = [dm.dm_adamw_state(W0, s) for s in (dm.DM_STATE_FP32, dm.DM_STATE_8BIT)]
            ts = [dm.dm_adamw_tensor(W[k], G, *st[k]) for k in (0, 1)]
            hp = dm.dm_adamw_default_hparams()
            dm.check(dm.dm_adamw_step(ts, hp, workspace(ts, hp)))
            res.append((W, st))
        (Wa, Sa), (Wb, Sb) = res
        keep = torch.ones(n, dtype=torch.bool, device="cuda")
        keep[300] = False
        for k in (0, 1):
            assert torch.equal(Wa[k][keep], Wb[k][keep])
        assert torch.equal(Sa[0][0][keep], Sb[0][0][keep])
        assert not torch.isfinite(Sb[0][0][300]) and not torch.isfinite(Sb[0][1][300])
        blocks = torch.arange(8, device="cuda") != 300 // 128
        for k in (2, 3):
            assert torch.equal(Sa[1][k][blocks], Sb[1][k][blocks])
            assert torch.isnan(Sb[1][k][300 // 128])
        elems = torch.arange(n, device="cuda") // 128 != 300 // 128
        for k in (0, 1):
            assert torch.equal(Sa[1][k].view(torch.uint8)[elems], Sb[1][k].view(torch.uint8)[elems])


def test_extreme_gradients():
    """Gradients of 1e-30 and 1e15 next to ordinary ones, fp32 moments; and
    zeros everywhere (the update is 0 / eps)."""
    n = 4096
    rng = np.random.default_rng(7)
    G = rng.standard_normal(n) * np.repeat([1e-30, 1.0, 1e15, 0.0], n // 4)
    W, z = rng.standard_normal(n), np.zeros(n)
    for state in (dm.DM_STATE_FP32, dm.DM_STATE_8BIT):
        Wd, Gd = (torch.from_numpy(x).float().cuda() for x in (W, G))
        st = dm.dm_adamw_state(Wd, state)
        hp = dm.dm_adamw_default_hparams(weight_decay=0.0)
        ts = [dm.dm_adamw_tensor(Wd, Gd, *st)]
        dm.check(dm.dm_adamw_step(ts, hp, workspace(ts, hp)))
        W0, G0 = W.astype(np.float32).astype(float), G.astype(np.float32).astype(float)
        out = to_host(Wd)
        # squares of 1e-30 underflow fp32: the update's divisor is then eps alone,
        # and the oracle's sqrt(v) = 1e-30 vanishes next to eps as well
        check_fp32(W0, G0, z, z, hp, 1, out, None, None, F32)
        assert np.array_equal(out[-n // 4:], W0[-n // 4:])


@pytest.mark.parametrize("state", [dm.DM_STATE_FP32, dm.DM_STATE_8BIT])
@pytest.mark.parametrize("eps", [0.0, 1e-30])
def test_tiny_eps_divides_by_subnormal_moments(state, eps):
    """Gradients whose second moments are subnormal (1e-40): with eps next to
    nothing the first step is still lr times the sign.  v = 1e-3 g^2 in steps of
    2^-149 is off by half a step, 2^-150 / 1e-40 relative: the update by half of that."""
    n = 1000
    g = torch.full((n,), 10.0 ** -18.5, device="cuda")
    g[::2] *= -1
    W = torch.zeros(n, device="cuda")
    st = dm.dm_adamw_state(W, state)
    hp = dm.dm_adamw_default_hparams(lr=0.5, weight_decay=0.0, eps=eps)
    ts = [dm.dm_adamw_tensor(W, g, *st)]
    dm.check(dm.dm_adamw_step(ts, hp, workspace(ts, hp)))
    want = -0.5 * np.sign(to_host(g))
    # g^2 = 1e-37 is normal; its product with 1e-3 rounds to a multiple of 2^-149
    assert np.all(np.abs(to_host(W) - want) <= 0.5 * (16 * U + 0.5 * 2.0 ** -150 / 1e-40))


@pytest.mark.parametrize("state", [dm.DM_STATE_FP32, dm.DM_STATE_8BIT])
def test_counted_steps_in_a_graph_equal_eager_steps(state):
    """A captured step with a device counter and learning rate, replayed, does
    what host-counted steps do, bit for bit."""
    n = 3001
    torch.manual_seed(0)
    W0 = torch.randn(n, device="cuda")
    grads = [torch.randn(n, device="cuda") for _ in range(4)]
    lrs = [1e-3, 2e-3, 5e-4, 1e-3]
    We = W0.clone()
    se = dm.dm_adamw_state(We, state)
    hp = dm.dm_adamw_default_hparams(seed=3, weight_decay=0.1)
    G = grads[0].clone()
    ts = [dm.dm_adamw_tensor(We, G, *se)]
    ws = workspace(ts, hp)
    for t in range(4):
        G.copy_(grads[t])
        hp.step, hp.lr = t + 1, lrs[t]
        dm.check(dm.dm_adamw_step(ts, hp, ws))
    Wg = W0.clone()
    sg = dm.dm_adamw_state(Wg, state)
    counter = torch.zeros(1, dtype=torch.int64, device="cuda")
    lr = torch.zeros(1, device="cuda")
    hg = dm.dm_adamw_default_hparams(seed=3, weight_decay=0.1, step_counter=counter, lr_dev=lr)
    tg = [dm.dm_adamw_tensor(Wg, G, *sg)]
    wg = workspace(tg, hg)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dm.check(dm.dm_adamw_step(tg, hg, wg))
    assert counter.item() == 0
    for t in range(4):
        G.copy_(grads[t])
        lr.fill_(lrs[t])
        graph.replay()
    torch.cuda.synchronize()
    assert counter.item() == 4 and dm.dm_read_device_status(wg) == dm.DM_OK
    assert torch.equal(We, Wg)
    for a, b in zip(se, sg):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_on_another_stream():
    n = 1 << 20
    s = torch.cuda.Stream()
    W, G = torch.randn(n, device="cuda"), torch.randn(n, device="cuda")
    st = dm.dm_adamw_state(W)
    h = [to_host(x) for x in (W, G, *st)]
    hp = dm.dm_adamw_default_hparams()
    ts = [dm.dm_adamw_tensor(W, G, *st)]
    ws = workspace(ts, hp)
    s.wait_stream(torch.cuda.current_stream())
    dm.check(dm.dm_adamw_step(ts, hp, ws, stream=s))
    assert dm.dm_read_device_status(ws, stream=s) == dm.DM_OK
    check_fp32(*h, hp, 1, to_host(W), to_host(st[0]), to_host(st[1]), F32)


def test_descriptors_keep_their_tensors():
    """Moments made in the descriptor's call live as long as the descriptors:
    memory allocated afterwards is other memory."""
    W, G = torch.zeros(5000, device="cuda"), torch.ones(5000, device="cuda")
    for state in (dm.DM_STATE_FP32, dm.DM_STATE_8BIT):
        for ts in ([dm.dm_adamw_tensor(W, G, *dm.dm_adamw_state(W, state))],
                   dm.dm_adamw_tensors([dm.dm_adamw_tensor(W, G, *dm.dm_adamw_state(W, state))])):
            used = {ts[0].moment1, ts[0].moment2, ts[0].scale1, ts[0].scale2}
            fresh = [torch.empty(n, dtype=torch.uint8, device="cuda")
                     for n in (1024, 5000, 20000, 160) * 8]
            assert not used & {t.data_ptr() for t in fresh}
    cl = dm.dm_grad_tensors([dm.dm_grad_tensor(torch.ones(5000, device="cuda"))])
    assert cl[0].grad not in {torch.empty(20000, dtype=torch.uint8, device="cuda").data_ptr()
                              for _ in range(4)}


def test_nothing_to_do():
    hp = dm.dm_adamw_default_hparams()
    for ts in ([], [dm.dm_adamw_tensor(*(torch.zeros(0, device="cuda") for _ in range(4)))]):
        ws = workspace(ts, hp)
        dm.check(dm.dm_adamw_step(ts, hp, ws))
        assert dm.dm_read_device_status(ws) == dm.DM_OK


def test_other_device_values_are_refused():
    w = torch.zeros(8, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        dm.dm_adamw_tensor(torch.zeros(8, 8, device="cuda").t()[:2], *(
            torch.zeros(16, device="cuda") for _ in range(3)))
    with pytest.raises(ValueError, match="CUDA"):
        dm.dm_adamw_tensor(w, torch.zeros(8), w.clone(), w.clone())


@pytest.mark.slow
@pytest.mark.parametrize("state", [dm.DM_STATE_FP32, dm.DM_STATE_8BIT])
def test_offsets_past_32_bits(state):
    """A tensor of 2^32 + 5000 elements: both ends against the oracle, and the
    middle moved (every element has a gradient of one)."""
    n = (1 << 32) + 5000
    W = torch.zeros(n, dtype=BF, device="cuda")
    G = torch.ones(n, dtype=BF, device="cuda")
    st = dm.dm_adamw_state(W, state)
    k = 10000
    a, b, c, d = draw(k, 77)
    for part in (slice(0, k), slice(n - k, n)):
        W[part].copy_(torch.from_numpy(a))
        G[part].copy_(torch.from_numpy(b))
    hp = dm.dm_adamw_default_hparams(seed=11)
    p = ao.AdamWParams(hp.lr, hp.beta1, hp.beta2, hp.eps, hp.weight_decay)
    h = [(to_host(W[s]), to_host(G[s])) for s in (slice(0, k), slice(n - k, n))]
    ts = [dm.dm_adamw_tensor(W, G, *st)]
    dm.check(dm.dm_adamw_step(ts, hp, workspace(ts, hp)))
    z = np.zeros(k)
    for s, (w0, g0), first in ((slice(0, k), h[0], 0), (slice(n - k, n), h[1], n - k)):
        check_fp32(w0, g0, z, z, hp, 1, to_host(W[s]), None, None, BF)
        if state == dm.DM_STATE_FP32:
            m32, v32 = ao.moments_f32(g0, z, z, p)
            assert np.array_equal(to_host(st[0][s]), m32) and np.array_equal(to_host(st[1][s]), v32)
            continue
        # whole blocks of the tail: its last 5000 elements start on a block's edge
        q = k - 5000 if first else 0
        m32, v32 = (x[q:q + 4992].astype(float) for x in ao.moments_f32(g0, z, z, p))
        u1, u2 = ao.noise(11, 1, 0, 4992, first=first + q)
        s1, s2 = ao.block_scales(m32, 448.0), ao.block_scales(v32, 57344.0)
        c1 = ao.stochastic_codes(m32, s1, ao.E4M3, u1) + 128 * np.signbit(m32)
        assert np.array_equal(st[0][first + q:first + q + 4992].view(torch.uint8).cpu().numpy(), c1)
        bl = (first + q) // 128
        assert np.array_equal(to_host(st[2][bl:bl + 39]), s1)
        assert np.array_equal(to_host(st[3][bl:bl + 39]), s2)
    mid = W[k:n - k]
    assert (mid < 0).all()
